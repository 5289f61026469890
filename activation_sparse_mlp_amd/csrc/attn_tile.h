// Attention of drafted tokens over the paged cache (gfx950, wave64).
//
//   score(c, j) = scale q_c . k_j,  o_c = sum_j softmax_j(score(c, .)) v_j
//
// A "column" c is one query head of one drafted token; the columns that share
// a kv head (tokens x heads per kv head) are computed together, so each key and
// value is read from HBM once per column tile group (up to 128 columns).
//
// Split.  The work is cut into steps of TS tokens (32 fp16, 64 fp8) of a unit
// (request, kv head, column tile group), and the steps of all units, laid end
// to end, are dealt to the workgroups in equal contiguous shares.  So one long
// request fills the chip as well as many short ones, ragged batches balance by
// themselves, and nothing has to be known on the host: each workgroup sums the
// lengths for itself.  A workgroup that does not cover a whole unit writes its
// running maximum, sum and unnormalised output to a slot of the workspace
// (at most two slots per workgroup), and a second launch joins a unit's slots in
// order; a unit inside one workgroup is stored at once.
//
// Matrix products, both with the columns as the B operand (16 per instruction):
//   S^T = K Q^T   A operand: 16 tokens x 32 dimensions, a lane's 16-byte packet
//                 is 8 (16) dimensions of one token;
//   O^T += V^T P^T  A operand: 16 dimensions x 32 tokens, a lane's packet is 8
//                 (16) tokens of one dimension.
// The cache's packet layout makes both loads 256 contiguous bytes per 16 lanes,
// whole cache lines straight into registers, with no transposition and no LDS.
// (Token rows picked so that the weights came out of the first product where the
// second wants them would read half lines, twice each: the cache then stalls on
// its own misses, 0.63 us a request instead of 0.2.)  A lane's scores are tokens
// 16 t + 4 g + i; the second product wants E g + e: a transposition of four-token
// groups among the four rows of lanes, two lane swaps per register of weights.
//
// Precision.  fp32 queries are split in hi + lo halves after a power-of-two
// scale per column, the softmax weights likewise (2^6 above the running
// maximum's, so that lo keeps its bits): fp32 in, fp32 out, errors near fp32's.
// With at most 8 columns hi and lo share one instruction (columns 0..7 and
// 8..15), otherwise they take one each into the same accumulator.  fp16 queries
// (fp16 out) are used as they are, their weights rounded once to fp16.  Scores,
// maxima, sums and outputs stay fp32 in registers.
//
// The running maximum is only raised when some score of the wave passes it by
// 2^8 (one vote), so the usual step neither exchanges lanes nor rescales.
#pragma once

#include "device.h"

namespace spffn {
namespace attn {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

constexpr float kNegInf = -__builtin_inff();
constexpr int kThreads = 256;

// Beginning and ending a unit costs a workgroup about as much time as this many
// steps, so a unit counts for as many more when the work is dealt out (a share
// that ends within them leaves the unit to the next workgroup).  Sixteen ragged
// requests of 96 heads: 397 us with 0, 313 with 4, 287 with 8 and with 16.
constexpr int kSetup = 8;

// A share is at least this many steps: with less, starting more workgroups and
// joining more parts costs more than it saves (one request of 4096 tokens and 8
// kv heads: 18.1 us with 4, 15.4 with 8, 19.0 with 16).
constexpr int kMinShare = 8;

enum Mode : int { kHalf = 0, kOne = 1, kTwo = 2 };  // columns per wave: 8, 16, 32

// What the second launch has to join for a workgroup of the first: its unit,
// and (an array of its own) of how many workgroups after it the unit has parts.
struct Task {
    int a0, n_cols, h, qt;
};

struct Args {
    const void *q;
    void *out;
    const uint8_t *k, *v;
    const float *ks, *vs;
    const int32_t *starts, *lens, *table;
    const int64_t *mask;
    float *part_o, *part_ml;
    Task *tasks;
    int *more;
    int64_t ldq, ldo;
    float scale;
    int N, R, G, H, width, pages, shift, max_new;
    int narrow;  // R <= 64 and every position fits 31 bits
    int wq;  // waves along the columns (1, 2, 4); 4 / wq along the tokens
    bool clear;  // the join kernel writes zeros to the rows that no request names
};

// What a request asks for: committed length L, tokens T, keys tot = L + T.
struct Req {
    int a0, L, T, tot, steps, span, nqt;
};

template <int TS>
__device__ __forceinline__ Req request(const Args &a, int r, int cw) {
    Req q;  // (r may differ between lanes)
    int a0 = a.starts[r], a1 = a.starts[r + 1];
    a0 = a0 < 0 ? 0 : a0;
    a1 = a1 > a.N ? a.N : a1;
    int T = a1 - a0;
    T = T < 0 ? 0 : T > a.max_new ? a.max_new : T;
    const int64_t cap64 = (int64_t)a.width << a.shift;
    const int cap = cap64 > 0x7FFFFF00 ? 0x7FFFFF00 : (int)cap64;
    int L = a.lens[r];
    L = L < 0 ? 0 : L > cap ? cap : L;
    q.a0 = a0;
    q.L = L;
    q.T = T;
    q.tot = cap - L < T ? cap : L + T;
    q.steps = (q.tot + TS - 1) / TS;
    q.span = q.steps + kSetup;
    q.nqt = (T * a.G + cw - 1) / cw;
    return q;
}

// Steps of request r over all its units.
template <int TS>
__device__ __forceinline__ int64_t req_steps(const Args &a, int r, int cw) {
    if (r >= a.R) return 0;
    const Req q = request<TS>(a, r, cw);
    return (int64_t)q.span * q.nqt * a.H;
}

__device__ __forceinline__ int64_t scan64(int64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t u = __shfl_up(v, o, 64);
        if (lane >= o) v += u;
    }
    return v;
}

// A value that every lane holds, in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)uniform((int)(uint32_t)v) |
                     (uint64_t)(uint32_t)uniform((int)((uint64_t)v >> 32)) << 32);
}

__device__ __forceinline__ Req uniform(const Req &q) {
    return Req{uniform(q.a0), uniform(q.L), uniform(q.T), uniform(q.tot), uniform(q.steps),
               uniform(q.span), uniform(q.nqt)};
}

// Inclusive sum over the lanes, by lane shifts within rows of 16 and two
// broadcasts across them.
__device__ __forceinline__ int scan32(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31
    return v;
}

// Every wave computes the plan for itself: the total and each workgroup's share.
template <int TS>
__device__ __forceinline__ int64_t plan_total(const Args &a, int cw, int lane, int64_t &incl0) {
    if (a.narrow) {  // up to 64 requests, their sum in 32 bits
        const int incl = scan32((int)req_steps<TS>(a, lane, cw));
        incl0 = incl;
        return __builtin_amdgcn_readlane(incl, 63);
    }
    int64_t total = 0;
    for (int b = 0; b < a.R; b += 64) {
        const int64_t incl = scan64(req_steps<TS>(a, b + lane, cw), lane);
        if (b == 0) incl0 = incl;
        total += __shfl(incl, 63, 64);
    }
    return uniform(total);
}

// The request that holds position p < total, and its first position.
template <int TS>
__device__ __forceinline__ int plan_find(const Args &a, int cw, int lane, int64_t incl0, int64_t p,
                                         int64_t &base) {
    if (a.narrow) {
        const int incl = (int)incl0;
        const int i = __ffsll((long long)__ballot((int)p < incl)) - 1;
        base = i ? __builtin_amdgcn_readlane(incl, i - 1) : 0;
        return i;
    }
    int64_t before = 0;
    for (int b = 0; b < a.R; b += 64) {
        const int64_t incl =
            before + (b == 0 ? incl0 : scan64(req_steps<TS>(a, b + lane, cw), lane));
        const uint64_t past = __ballot(p < incl);
        if (past) {
            const int i = __ffsll((long long)past) - 1;
            base = uniform(i ? __shfl(incl, i - 1, 64) : before);
            return uniform(b + i);
        }
        before = __shfl(incl, 63, 64);
    }
    base = 0;  // not reached for p < total
    return 0;
}

constexpr int kMaxWgs = 768;  // of a launch

// Steps per workgroup, a multiple of the waves along the tokens (a power of two).
template <int WGS>
__device__ __forceinline__ int64_t share(int64_t total, int wk) {
    const int64_t c = (int64_t)((uint64_t)(total + WGS - 1) / (uint64_t)WGS);
    if (c < kMinShare) return kMinShare;
    return (c + wk - 1) & ~(int64_t)(wk - 1);
}

// Eight dimensions (tokens) of a packet as halves.
__device__ __forceinline__ half8 fp8_half(uint32_t w0, uint32_t w1) {
    const half2v a = __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, false));
    const half2v b = __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, true));
    const half2v c = __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, false));
    const half2v d = __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, true));
    return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <bool FP8>
__device__ __forceinline__ half8 packet_half(const uint4 &p, int hf) {
    if constexpr (FP8) return hf ? fp8_half(p.z, p.w) : fp8_half(p.x, p.y);
    else return __builtin_bit_cast(half8, p);
}

// Nonzero where one of a word's elements (2 fp16, 4 fp8) is not finite.
template <bool FP8>
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) {
    if constexpr (FP8)  // 0x7F or 0xFF: adding 1 to the low seven bits carries into the eighth
        return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    else  // exponent all ones: adding one step of it carries into the sign's place
        return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
}

// The word with those elements zero.
template <bool FP8>
__device__ __forceinline__ uint32_t drop_odd(uint32_t w) {
    const uint32_t b = odd_bits<FP8>(w);
    if constexpr (FP8) return w & ~((b >> 7) * 0xFFu);
    else return w & ~((b >> 15) * 0xFFFFu);
}

__device__ __forceinline__ float over_groups_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float over_groups_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

template <bool ONCE>
__device__ __forceinline__ u32x4_t fetch(const uint8_t *p) {
    if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(p));
    else return *reinterpret_cast<const u32x4_t *>(p);
}

// Final value of one output element: o / l, 0 for a row that saw no key, NaN
// for one whose every key scored -inf.
__device__ __forceinline__ float finish(float o, float m, float l, float inv) {
    if (m == kNegInf) return l > 0.0f ? __builtin_nanf("") : l == 0.0f ? 0.0f : l;
    return o * inv;
}

struct Sum {
    float m, l;
    f32x4 o;
};

__device__ __forceinline__ void join(Sum &a, float m, float l, const f32x4 &o) {
    const float top = fmaxf(a.m, m);
    const float f0 = top == kNegInf ? 1.0f : exp2f(a.m - top);
    const float f1 = top == kNegInf ? 1.0f : exp2f(m - top);
    a.l = f0 * a.l + f1 * l;
    a.o = a.o * f0 + o * f1;
    a.m = top;
}

// Four dimensions, from `at` on, of column cg of kv head h.
template <bool Q16, int D>
__device__ __forceinline__ void store_out(const Args &a, int a0, int h, int cg, int at, const f32x4 &o,
                                          float m, float l, float inv) {
    const int t = cg / a.G, gq = cg - t * a.G;
    const size_t to = (size_t)(a0 + t) * a.ldo + (size_t)(h * a.G + gq) * D + at;
    if constexpr (Q16) {
        half4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (_Float16)finish(o[i], m, l, inv);
        *reinterpret_cast<half4 *>(static_cast<_Float16 *>(a.out) + to) = y;
    } else {
        f32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = finish(o[i], m, l, inv);
        *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + to) = y;
    }
}

// x's odd rows of 16 lanes with y's even rows; x's upper 32 lanes with y's lower.
__device__ __forceinline__ void swap16(uint2 &x, uint2 &y) {
    const auto a = __builtin_amdgcn_permlane16_swap(x.x, y.x, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(x.y, y.y, false, false);
    x = make_uint2(a[0], b[0]);
    y = make_uint2(a[1], b[1]);
}
__device__ __forceinline__ void swap32(uint2 &x, uint2 &y) {
    const auto a = __builtin_amdgcn_permlane32_swap(x.x, y.x, false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(x.y, y.y, false, false);
    x = make_uint2(a[0], b[0]);
    y = make_uint2(a[1], b[1]);
}

// Weights of tokens 16 t + 4 g + i (register t, lane row g) to the B operand's
// tokens E g + e.
__device__ __forceinline__ void to_packets(uint2 (&w)[2], half8 (&p)[1]) {
    swap32(w[0], w[1]);
    swap16(w[0], w[1]);
    p[0] = __builtin_bit_cast(half8, make_uint4(w[0].x, w[0].y, w[1].x, w[1].y));
}
__device__ __forceinline__ void to_packets(uint2 (&w)[4], half8 (&p)[2]) {
    swap32(w[0], w[2]);
    swap32(w[1], w[3]);
    swap16(w[0], w[1]);
    swap16(w[2], w[3]);
    p[0] = __builtin_bit_cast(half8, make_uint4(w[0].x, w[0].y, w[1].x, w[1].y));
    p[1] = __builtin_bit_cast(half8, make_uint4(w[2].x, w[2].y, w[3].x, w[3].y));
}

template <bool FP8, bool Q16, int D, int MODE>
struct Cfg {
    static constexpr int E = FP8 ? 16 : 8;
    static constexpr int TS = 4 * E;               // tokens per step
    static constexpr int TT = TS / 16;             // token tiles per step
    static constexpr int HF = E / 8;               // instructions per packet
    static constexpr int NPK = D / E;              // packets per token
    static constexpr int KP = (NPK + 3) / 4;       // packets per lane and tile
    static constexpr int KS = KP * HF;             // instructions per tile
    static constexpr int DT = D / 16;              // dimension tiles
    static constexpr int NQ = MODE == kTwo ? 2 : 1;
    static constexpr bool HALF = MODE == kHalf;
    static constexpr bool SPLIT = !Q16;            // hi + lo
    static constexpr bool LO = SPLIT && !HALF;     // lo takes instructions of its own
    static constexpr int PL = LO ? 2 : 1;          // planes of queries
    static constexpr bool QLDS = MODE == kTwo;     // queries in LDS, to leave registers
    static constexpr int QBYTES = QLDS ? 4 * PL * NQ * KS * 1024 : 0;
    static constexpr int COLS = HALF ? 8 : 16 * NQ;  // columns per wave
    static constexpr int PITCH = D + 4;
    // waves per SIMD the registers have to leave room for
    static constexpr int WAVES = D > 128 ? 1 : MODE == kTwo || D > 96 ? 2 : 3;
    static constexpr int WGS = 256 * WAVES;  // workgroups of a launch: all resident at once
    // a step's keys and values are read once by one wave: past the caches, then
    static constexpr bool ONCE = MODE != kTwo;
};

template <bool FP8, bool Q16, int D, int MODE>
__global__ __launch_bounds__(kThreads, (Cfg<FP8, Q16, D, MODE>::WAVES)) void attend_kernel(Args a) {
    using C = Cfg<FP8, Q16, D, MODE>;
    constexpr int E = C::E, TS = C::TS, TT = C::TT, HF = C::HF, KP = C::KP, DT = C::DT, NQ = C::NQ;
    constexpr uint32_t kAll = (1u << E) - 1u;
    extern __shared__ __align__(16) float lds[];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int WQ = a.wq, WK = 4 / WQ;
    const int wq = wv & (WQ - 1), wk = wv / WQ;
    const int cw = C::COLS * WQ;
    const int ps = 1 << a.shift;

    int64_t incl0 = 0, base;
    const int64_t total = plan_total<TS>(a, cw, lane, incl0);
    const int64_t per = share<C::WGS>(total, WK);
    int64_t p = (int64_t)blockIdx.x * per;
    const int64_t end = p + per < total ? p + per : total;
    int more = 0;
    if (p >= end) {
        if (threadIdx.x == 0) a.more[blockIdx.x] = 0;
        return;
    }
    int r = plan_find<TS>(a, cw, lane, incl0, p, base);

    Req rq = uniform(request<TS>(a, r, cw));
    int64_t rsteps = (int64_t)rq.span * rq.nqt * a.H;
    while (true) {
        // ---- the segment: steps [s0, s1) of unit (r, h, qt) ----
        const uint32_t rel = (uint32_t)(p - base);
        const uint32_t unit = (uint32_t)uniform((int)(rel / (uint32_t)rq.span));
        const int x0 = (int)(rel - unit * (uint32_t)rq.span);  // its place in the unit's span
        const int x1 = end - p < rq.span - x0 ? x0 + (int)(end - p) : rq.span;
        if (x1 <= kSetup) break;  // the share's end: the unit is the next workgroup's
        const int s0 = x0 > kSetup ? x0 - kSetup : 0, s1 = x1 - kSetup;
        const int h = uniform((int)(unit / (uint32_t)rq.nqt)), qt = (int)(unit - (uint32_t)h * rq.nqt);
        const int n_cols = rq.T * a.G;
        const int col0 = (qt * WQ + wq) * C::COLS;
        const int32_t *trow = a.table + (size_t)r * a.width;

        // A step covers TT blocks of 16 tokens, each on one page: lane b (mod TT) holds block b's.
        // No load here hangs on a condition: one that may be skipped would make the loads
        // behind it be waited for as if it had been.  What is not wanted is read twice.
        auto pages_of = [&](int st) {
            const int tok = st * TS + 16 * (lane & (TT - 1));
            const int pg = trow[(tok < rq.tot ? tok : rq.tot - 1) >> a.shift];
            return tok < rq.tot ? pg : -1;
        };
        auto next = [&](int st) { return st + WK < s1 ? st + WK : st; };
        int st = s0 + wk;
        const int first = st < s1 ? st : s1 - 1;  // (a wave without a step reads and drops one)
        int pg0 = pages_of(first), pg1 = pages_of(next(first));  // pages of this step and the next

        // ---- queries as B operands ----
        half8 qr[C::QLDS ? 1 : C::PL][C::QLDS ? 1 : NQ][C::QLDS ? 1 : C::KS];
        half8 *qs = reinterpret_cast<half8 *>(lds) + (size_t)wv * (C::QBYTES / 64) + lane;
        auto q_put = [&](int p, int j, int i, const half8 &x) {
            if constexpr (C::QLDS) qs[((p * NQ + j) * C::KS + i) * 64] = x;
            else qr[p][j][i] = x;
        };
        auto q_get = [&](int p, int j, int i) {
            if constexpr (C::QLDS) return qs[((p * NQ + j) * C::KS + i) * 64];
            else return qr[p][j][i];
        };
        float cf[NQ];
        uint64_t bits[NQ];
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int c = col0 + (C::HALF ? (n & 7) : j * 16 + n);
            const bool real = c < n_cols;
            const int t = real ? c / a.G : 0, gq = real ? c - t * a.G : 0;
            const int row = rq.a0 + t;
            bits[j] = 0;
            if (real) {
                bits[j] = a.mask ? (uint64_t)a.mask[row] : (~0ull >> (63 - t));
                const int tk = rq.tot - rq.L;
                bits[j] &= tk <= 0 ? 0ull : (~0ull >> (64 - tk));
            }
            // scores are compared before they are scaled: the factor is kept positive
            const float unit_scale =
                fabsf(a.scale) * 1.44269504088896340736f * (FP8 ? fabsf(a.ks[h]) : 1.0f);
            const bool flip = (a.scale < 0.0f) != (FP8 && a.ks[h] < 0.0f);
            const size_t at = (size_t)row * a.ldq + (size_t)(h * a.G + gq) * D;
            if constexpr (Q16) {
                const _Float16 *qp = static_cast<const _Float16 *>(a.q) + at;
#pragma unroll
                for (int i = 0; i < C::KS; ++i) {
                    const int d = ((i / HF) * 4 + g) * E + (i % HF) * 8;
                    half8 x = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (real && d < D) x = *reinterpret_cast<const half8 *>(qp + d);
                    if (flip) x = -x;
                    q_put(0, j, i, x);
                }
                cf[j] = unit_scale;
            } else {
                const float *qp = static_cast<const float *>(a.q) + at;
                float x[C::KS][8];
                float m = 0.0f, odd = 0.0f;
#pragma unroll
                for (int i = 0; i < C::KS; ++i) {
                    const int d = ((i / HF) * 4 + g) * E + (i % HF) * 8;
                    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), w = u;
                    if (real && d < D) {
                        u = *reinterpret_cast<const float4 *>(qp + d);
                        w = *reinterpret_cast<const float4 *>(qp + d + 4);
                    }
                    x[i][0] = u.x; x[i][1] = u.y; x[i][2] = u.z; x[i][3] = u.w;
                    x[i][4] = w.x; x[i][5] = w.y; x[i][6] = w.z; x[i][7] = w.w;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        m = fmaxf(m, fabsf(x[i][e]));
                        odd += x[i][e] * 0.0f;  // NaN as soon as one value is not finite
                    }
                }
                m = over_groups_max(m);
                odd = over_groups_sum(odd);
                uint32_t eb = __float_as_uint(m) >> 23;
                eb = eb < 16 ? 16 : eb > 254 ? 254 : eb;
                const float up = __uint_as_float((267u - eb) << 23 | (flip ? 1u << 31 : 0u));  // to [2^13, 2^14)
                // a query that is not finite makes every score NaN
                cf[j] = unit_scale * __uint_as_float((eb - 13u) << 23) + odd;
#pragma unroll
                for (int i = 0; i < C::KS; ++i) {
                    half8 hi, lo;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float v = x[i][e] * up;
                        hi[e] = (_Float16)v;
                        lo[e] = (_Float16)(v - (float)hi[e]);
                    }
                    if constexpr (C::HALF) {
                        q_put(0, j, i, n < 8 ? hi : lo);
                    } else {
                        q_put(0, j, i, hi);
                        q_put(1, j, i, lo);
                    }
                }
            }
        }

        f32x4 o[NQ][DT];
        float ref[NQ], l[NQ];
        bool seen[NQ];
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            ref[j] = kNegInf;
            l[j] = 0.0f;
            seen[j] = false;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[j][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        // ---- the steps of this wave.  Keys of the next step are requested as soon as this
        // step's scores are taken, its values as soon as this step's have been used, its page
        // numbers a step earlier still: every load has half a step or more to arrive.
        const int tvl = g * E;  // first token of a lane's value packet
        const uint32_t klane = (((uint32_t)g << a.shift) + n) * 16;  // bytes within a tile's keys
        const uint8_t *kbase = a.k + (size_t)h * ((size_t)C::NPK << a.shift) * 16;
        const uint8_t *vbase = a.v + ((size_t)h * (ps / E) * D + n) * 16;
        const uint64_t kstride = (uint64_t)a.H * ((size_t)C::NPK << a.shift) * 16;  // bytes per page
        const uint64_t vstride = (uint64_t)a.H * (ps / E) * D * 16;
        u32x4_t kp[TT][KP], vp[DT];
        auto there = [&](int pg) { return (uint32_t)pg < (uint32_t)a.pages; };
        auto load_k = [&](int st, int pgs) {  // a page that is not there reads page 0 (and is masked)
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int pg = __builtin_amdgcn_readlane(pgs, t);
                const uint8_t *kb = kbase + (uint64_t)(there(pg) ? pg : 0) * kstride +
                                    (uint32_t)((st * TS + 16 * t) & (ps - 1)) * 16;
#pragma unroll
                for (int i = 0; i < KP; ++i) {
                    // a packet past the head's meets queries of 0: the lane's one before is as good
                    const bool real = C::NPK % 4 == 0 || i * 4 + g < C::NPK;
                    kp[t][i] =
                        fetch<C::ONCE>(kb + ((uint32_t)((real ? i : i - 1) * 64) << a.shift) + klane);
                }
            }
        };
        auto load_v = [&](int st, int pgs) {
            uint64_t off = 0;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int pg = __builtin_amdgcn_readlane(pgs, t);
                const uint64_t x = (uint64_t)(there(pg) ? pg : 0) * vstride;
                if (t == 0 || t == g * E / 16) off = x;
            }
            const uint8_t *vb =
                vbase + off + (uint32_t)((((st * TS + tvl) & (ps - 1)) / E) * D) * 16;
#pragma unroll
            for (int d = 0; d < DT; ++d) vp[d] = fetch<C::ONCE>(vb + d * 256);
        };
        __builtin_amdgcn_sched_barrier(0);  // in this order, or the loop waits for both at once
        load_k(first, pg0);
        __builtin_amdgcn_sched_barrier(0);
        load_v(first, pg0);
        __builtin_amdgcn_sched_barrier(0);
        for (; st < s1; st += WK) {
            const int st1 = next(st);
            const int t0 = st * TS, tv = t0 + tvl;
            const bool masked = t0 + TS > rq.L || __any(!there(pg0));
            const int pg2 = pages_of(next(st1));

            // ---- scores (unscaled) ----
            f32x4 s[NQ][TT];
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int j = 0; j < NQ; ++j) s[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < C::KS; ++i) {
                // queries from LDS: no more than two instructions' worth at a time
                if (C::QLDS && i % 2 == 0) __builtin_amdgcn_sched_barrier(0);
                half8 qx[NQ], qy[NQ];
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    qx[j] = q_get(0, j, i);
                    if constexpr (C::LO) qy[j] = q_get(1, j, i);
                }
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const half8 kx = packet_half<FP8>(__builtin_bit_cast(uint4, kp[t][i / HF]), i % HF);
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        s[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kx, qx[j], s[j][t], 0, 0, 0);
                        if constexpr (C::LO)
                            s[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kx, qy[j], s[j][t], 0, 0, 0);
                    }
                }
            }
            load_k(st1, pg1);
            if constexpr (C::HALF) {
                // columns n and n + 8 hold the products with hi and lo: add them
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[0][t][i] += __int_as_float(__builtin_amdgcn_mov_dpp(
                            __float_as_int(s[0][t][i]), 0x128, 0xF, 0xF, true));  // row_ror:8
            }

            // ---- masks ----
            uint32_t hid[NQ];  // bit 4t + i: token t0 + 16t + 4g + i does not count for this column
#pragma unroll
            for (int j = 0; j < NQ; ++j) hid[j] = 0;
            bool odd = false;  // some value of this step is not finite
            if (masked) {
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const int jt = t0 + 16 * t + 4 * g - rq.L;  // first one's place in the step's own
                    const uint32_t old = jt >= 0 ? 0u : jt <= -4 ? 15u : (1u << -jt) - 1u;
                    const bool on_page = there(__builtin_amdgcn_readlane(pg0, t));
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        const uint64_t own = jt >= 64 || jt <= -4 ? 0ull
                                             : jt >= 0 ? bits[j] >> jt : bits[j] << -jt;
                        hid[j] |= (on_page ? ~(old | (uint32_t)own) & 15u : 15u) << (4 * t);
                    }
                }
#pragma unroll
                for (int j = 0; j < NQ; ++j)
#pragma unroll
                    for (int t = 0; t < TT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if ((hid[j] >> (4 * t + i)) & 1) s[j][t][i] = kNegInf;
                // values behind the last token or on no page are whatever memory holds: out
                const bool ok_v = there(__shfl(pg0, g * E / 16, 64));
                const int left = ok_v ? rq.tot - tv : 0;
                uint32_t keep[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int n_in = left - w * (E / 4);  // tokens of this word that are there
                    keep[w] = n_in >= E / 4 ? ~0u : n_in <= 0 ? 0u : (1u << (n_in * (128 / E))) - 1u;
                }
                uint32_t worst = 0;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        vp[d][w] &= keep[w];
                        worst |= odd_bits<FP8>(vp[d][w]);
                    }
                odd = __any(worst != 0);
                if (odd) {
                    // values that are not finite leave the product too (a weight of 0 would
                    // make NaN of them) and are added at the end
#pragma unroll
                    for (int d = 0; d < DT; ++d)
#pragma unroll
                        for (int w = 0; w < 4; ++w) vp[d][w] = drop_odd<FP8>(vp[d][w]);
                }
            }

            // ---- softmax weights ----
            half8 ph[NQ][HF], pl[C::LO ? NQ : 1][HF];
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                float top = s[j][0][0];
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, s[j][t][i]);
                top *= cf[j];
                if (__any(top > ref[j] + 8.0f)) {
                    const float up = fmaxf(ref[j], over_groups_max(top));
                    const float alpha = up == kNegInf ? 1.0f : exp2f(ref[j] - up);
                    l[j] *= alpha;
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        __builtin_amdgcn_sched_barrier(0);  // a tile at a time: few registers
                        o[j][d] *= alpha;
                    }
                    ref[j] = up;
                }
                seen[j] = seen[j] || hid[j] != kAll;
                const float sub = 6.0f - (ref[j] == kNegInf ? 0.0f : ref[j]);
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[j][t][i] = __builtin_amdgcn_exp2f(fmaf(s[j][t][i], cf[j], sub));
                if (masked) {  // (a scale of 0 makes a hidden score NaN, not -inf)
#pragma unroll
                    for (int t = 0; t < TT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if ((hid[j] >> (4 * t + i)) & 1) s[j][t][i] = 0.0f;
                }
                uint2 wh[TT], wl[TT];  // four weights each
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    half4 hi, lo;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float w = s[j][t][i];
                        hi[i] = (_Float16)w;
                        if constexpr (!Q16) {
                            lo[i] = (_Float16)(w - (float)hi[i]);
                            l[j] += w;
                        }
                        if constexpr (C::HALF) hi[i] = n < 8 ? hi[i] : lo[i];
                    }
                    wh[t] = __builtin_bit_cast(uint2, hi);
                    if constexpr (C::LO) wl[t] = __builtin_bit_cast(uint2, lo);
                }
                to_packets(wh, ph[j]);
                if constexpr (C::LO) to_packets(wl, pl[j]);
                if constexpr (Q16) {
                    // the sum of the weights as they are used, by a product with ones
                    f32x4 sum = {l[j], 0.f, 0.f, 0.f};
                    const _Float16 one = (_Float16)1.0f;
#pragma unroll
                    for (int hf = 0; hf < HF; ++hf)
                        sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            half8{one, one, one, one, one, one, one, one}, ph[j][hf], sum, 0, 0, 0);
                    l[j] = sum[0];
                }
            }

            // ---- outputs ----
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int hf = 0; hf < HF; ++hf) {
                    const half8 vx = packet_half<FP8>(__builtin_bit_cast(uint4, vp[d]), hf);
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        o[j][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vx, ph[j][hf], o[j][d], 0, 0, 0);
                        if constexpr (C::LO)
                            o[j][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vx, pl[j][hf], o[j][d], 0, 0, 0);
                    }
                }
            load_v(st1, pg1);
            if (odd) {
                // rare: the values that are not finite, one by one, for the columns that see them
                for (int tok = 0; tok < TS && t0 + tok < rq.tot; ++tok) {
                    const int gs = tok / E, e = tok % E;
                    const int pg = trow[(t0 + tok) >> a.shift];
                    if (!there(pg)) continue;
                    const size_t row = ((size_t)pg * a.H + h) * (ps / E) + ((t0 + tok) & (ps - 1)) / E;
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        float w = 0.0f;  // the weight's hi half: its sign and size are enough here
#pragma unroll
                        for (int x = 0; x < E; ++x)
                            if (x == e) w = (float)ph[j][x / 8][x % 8];
                        w = __shfl(w, gs * 16 + (C::HALF ? n & 7 : n), 64);
                        const int hx = __shfl((int)hid[j], ((tok >> 2) & 3) * 16 + n, 64);
                        const bool on = !((hx >> (4 * (tok >> 4) + (tok & 3))) & 1);
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            __builtin_amdgcn_sched_barrier(0);  // few registers, not few cycles
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const size_t at = (row * D + d * 16 + 4 * g + i) * E + e;
                                float v;
                                if constexpr (FP8)
                                    v = (a.v[at] & 0x7F) == 0x7F ? __builtin_nanf("") : 0.0f;
                                else v = (float)reinterpret_cast<const _Float16 *>(a.v)[at];
                                if (on && !(fabsf(v) < __builtin_inff())) o[j][d][i] += w * v;
                            }
                        }
                    }
                }
            }
            pg0 = pg1;
            pg1 = pg2;
        }

        // ---- the workgroup's share of the unit ----
        const bool whole = s0 == 0 && s1 == rq.steps;
        float vs = FP8 ? a.vs[h] : 1.0f;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            if constexpr (!Q16) l[j] = over_groups_sum(l[j]);
            const bool any = __shfl_xor(seen[j], 16, 64) || seen[j];
            seen[j] = __shfl_xor(any, 32, 64) || any;
            if (ref[j] == kNegInf && l[j] == 0.0f) l[j] = seen[j] ? 1.0f : 0.0f;
            if constexpr (C::HALF) {
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[j][d][i] += __int_as_float(__builtin_amdgcn_update_dpp(
                            0, __float_as_int(o[j][d][i]), 0x128, 0xF, 0xF, false));
            }
        }
        const size_t slot = 2 * (size_t)blockIdx.x + (s0 == 0 ? 1 : 0);
        if (!C::HALF && WK == 1) {
            // every wave has whole columns: straight from the registers
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                const int c = wq * C::COLS + j * 16 + n, cg = qt * cw + c;
                if (cg < n_cols) {
                    const float inv = vs / l[j];
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        const int at = d * 16 + 4 * g;
                        if (whole) store_out<Q16, D>(a, rq.a0, h, cg, at, o[j][d], ref[j], l[j], inv);
                        else *reinterpret_cast<f32x4 *>(a.part_o + (slot * cw + c) * D + at) = o[j][d];
                    }
                    if (!whole && g == 0) {
                        a.part_ml[(slot * cw + c) * 2] = ref[j];
                        a.part_ml[(slot * cw + c) * 2 + 1] = l[j];
                    }
                }
            }
        } else {
            // through LDS: [wave][column][D + 4], then maxima and sums [wave][column][2]
            if constexpr (C::QLDS) __syncthreads();  // every wave is done with its queries there
            float *lo_ = lds + (size_t)wv * C::COLS * C::PITCH;
            float *ml = lds + (size_t)4 * C::COLS * C::PITCH;
            if (!C::HALF || n < 8) {
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const int c = j * 16 + n;
#pragma unroll
                    for (int d = 0; d < DT; ++d)
                        *reinterpret_cast<f32x4 *>(lo_ + c * C::PITCH + d * 16 + 4 * g) = o[j][d];
                    if (g == 0) {
                        ml[(wv * C::COLS + c) * 2] = ref[j];
                        ml[(wv * C::COLS + c) * 2 + 1] = l[j];
                    }
                }
            }
            __syncthreads();
            for (int x = threadIdx.x; x < cw * (D / 4); x += kThreads) {
                const int c = x / (D / 4), d4 = x - c * (D / 4);
                const int w0 = c / C::COLS, cc = c - w0 * C::COLS;  // wave along the columns, its column
                const int cg = qt * cw + c;
                if (cg >= n_cols) break;
                Sum acc{kNegInf, 0.0f, f32x4{0.f, 0.f, 0.f, 0.f}};
                for (int kx = 0; kx < WK; ++kx) {
                    const int wx = kx * WQ + w0;
                    const float *p_ml = ml + (wx * C::COLS + cc) * 2;
                    join(acc, p_ml[0], p_ml[1],
                         *reinterpret_cast<const f32x4 *>(
                             lds + ((size_t)wx * C::COLS + cc) * C::PITCH + d4 * 4));
                }
                if (whole) {
                    store_out<Q16, D>(a, rq.a0, h, cg, d4 * 4, acc.o, acc.m, acc.l, vs / acc.l);
                } else {
                    *reinterpret_cast<f32x4 *>(a.part_o + (slot * cw + c) * D + d4 * 4) = acc.o;
                    if (d4 == 0) {
                        a.part_ml[(slot * cw + c) * 2] = acc.m;
                        a.part_ml[(slot * cw + c) * 2 + 1] = acc.l;
                    }
                }
            }
        }
        // a unit begun here and not finished: the workgroups after this one that go on with it
        if (s0 == 0 && !whole) {
            more = per >= rq.span - x1 ? 1 : (rq.span - x1 + (int)per - 1) / (int)per;
            if (threadIdx.x == 0) a.tasks[blockIdx.x] = Task{rq.a0, n_cols, h, qt};
        }

        // ---- next segment ----
        p += x1 - x0;
        if (p >= end) break;
        __syncthreads();  // the next segment reuses the LDS
        if (p - base >= rsteps) {
            do {
                base += rsteps;
                ++r;
                rq = uniform(request<TS>(a, r, cw));
                rsteps = (int64_t)rq.span * rq.nqt * a.H;
            } while (rsteps == 0);
        }
    }
    if (threadIdx.x == 0) a.more[blockIdx.x] = more;
}

// Joins the parts of the units that the attention launch dealt to several
// workgroups (its tasks): for a task of workgroup w, slot 2w + 1 holds the first
// part, the following workgroups' slots 2w' the rest.  Every workgroup gathers
// the tasks there are (at most one per workgroup of the first launch, usually
// one per unit) and takes its share of all their columns, JC at a time: a
// thread four outputs of a column and every JP-th part, four parts at a time so
// that their loads are in flight together; the JP sums of a column are then
// added in order.
constexpr int kJoinParts = 4;
constexpr int kJoinWgs = 1024;

template <bool FP8, bool Q16, int D>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(Args a, int wgs, int cw) {
    constexpr int JP = kJoinParts, TC = D / 4;  // threads per column and part group
    constexpr int JC = kThreads / (TC * JP);    // columns at a time
    __shared__ Sum part[JP][JC][TC];
    __shared__ uint16_t list[kMaxWgs];
    __shared__ int count[kMaxWgs / 64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    // ---- rows without a request, by the workgroups that get no task first ----
    if (a.clear)
        for (int row = gridDim.x - 1 - blockIdx.x; row < a.N; row += gridDim.x) {
            bool named = false;
            for (int r = threadIdx.x; r < a.R; r += kThreads) {
                const int from = max(a.starts[r], 0), to = min(a.starts[r + 1], a.N);
                named |= row >= from && row < to && row - from < a.max_new;
            }
            if (__syncthreads_or(named)) continue;
            for (int64_t i = threadIdx.x; i < (int64_t)a.H * a.G * D; i += kThreads) {
                if constexpr (Q16)
                    static_cast<_Float16 *>(a.out)[row * a.ldo + i] = (_Float16)0.0f;
                else
                    static_cast<float *>(a.out)[row * a.ldo + i] = 0.0f;
            }
        }
    // ---- the tasks, in order ----
    uint64_t have[kMaxWgs / kThreads];
#pragma unroll
    for (int k = 0; k < kMaxWgs / kThreads; ++k) {
        const int w = k * kThreads + threadIdx.x;
        have[k] = __ballot(w < wgs && a.more[w < wgs ? w : 0] > 0);
        if (lane == 0) count[k * (kThreads / 64) + wv] = __popcll(have[k]);
    }
    __syncthreads();
    int n_tasks = 0;
#pragma unroll
    for (int k = 0; k < kMaxWgs / kThreads; ++k) {
        int before = 0;
        for (int x = 0; x < k * (kThreads / 64) + wv; ++x) before += count[x];
        if ((have[k] >> lane) & 1)
            list[before + __popcll(have[k] & ((1ull << lane) - 1))] = (uint16_t)(k * kThreads + threadIdx.x);
    }
    for (int x = 0; x < kMaxWgs / 64; ++x) n_tasks += count[x];
    __syncthreads();
    // ---- a share of their columns ----
    const int rows = (cw + JC - 1) / JC;
    const int d4 = threadIdx.x % TC, jc = (threadIdx.x / TC) % JC, jp = threadIdx.x / (TC * JC);
    for (int item = blockIdx.x; item < n_tasks * rows; item += gridDim.x) {
        const int w = list[item / rows], c = item % rows * JC + jc;
        const Task task = a.tasks[w];
        const int more = a.more[w];
        const int cg = task.qt * cw + c;
        const bool real = c < cw && cg < task.n_cols && jp < JP;  // (96 dimensions leave threads over)
        Sum acc{kNegInf, 0.0f, f32x4{0.f, 0.f, 0.f, 0.f}};
        if (real) {
            for (int i = jp; i <= more; i += 4 * JP) {
                float m[4], l[4];
                f32x4 o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int x = i + k * JP <= more ? i + k * JP : i;
                    const size_t at = (size_t)(2 * (w + x) + (x == 0 ? 1 : 0)) * cw + c;
                    m[k] = a.part_ml[at * 2];
                    l[k] = a.part_ml[at * 2 + 1];
                    o[k] = *reinterpret_cast<const f32x4 *>(a.part_o + at * D + d4 * 4);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i + k * JP <= more) join(acc, m[k], l[k], o[k]);
            }
            part[jp][jc][d4] = acc;
        }
        __syncthreads();
        if (real && jp == 0) {
            const int parts = more + 1 < JP ? more + 1 : JP;
            for (int k = 1; k < parts; ++k)
                join(acc, part[k][jc][d4].m, part[k][jc][d4].l, part[k][jc][d4].o);
            store_out<Q16, D>(a, task.a0, task.h, cg, d4 * 4, acc.o, acc.m, acc.l,
                              (FP8 ? a.vs[task.h] : 1.0f) / acc.l);
        }
        __syncthreads();
    }
}

template <bool FP8, bool Q16, int D, int MODE>
hipError_t launch_mode(const Args &a, hipStream_t s) {
    using C = Cfg<FP8, Q16, D, MODE>;
    auto fn = attend_kernel<FP8, Q16, D, MODE>;
    size_t lds = (size_t)4 * C::COLS * (C::PITCH + 2) * 4;
    if (lds < (size_t)C::QBYTES) lds = C::QBYTES;
    if (lds > 65536) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    fn<<<C::WGS, kThreads, lds, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    attend_join_kernel<FP8, Q16, D><<<kJoinWgs, kThreads, 0, s>>>(a, C::WGS, C::COLS * a.wq);
    return hipGetLastError();
}

template <bool FP8, bool Q16, int D>
hipError_t launch_dim(const Args &a, int mode, hipStream_t s) {
    if constexpr (D <= 128)
        if (mode == kTwo) return launch_mode<FP8, Q16, D, kTwo>(a, s);
    if constexpr (!Q16)
        if (mode == kHalf) return launch_mode<FP8, Q16, D, kHalf>(a, s);
    return launch_mode<FP8, Q16, D, kOne>(a, s);
}

template <bool FP8, bool Q16>
hipError_t launch_all(const Args &a, int dim, int mode, hipStream_t s) {
    switch (dim) {
        case 64: return launch_dim<FP8, Q16, 64>(a, mode, s);
        case 96: return launch_dim<FP8, Q16, 96>(a, mode, s);
        case 128: return launch_dim<FP8, Q16, 128>(a, mode, s);
        default: return launch_dim<FP8, Q16, 256>(a, mode, s);
    }
}

}  // namespace attn
}  // namespace spffn
