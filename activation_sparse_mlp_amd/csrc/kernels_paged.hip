// The paged key/value cache: block tables and slot maps of a step, and the
// append of new rows.
//
// A cache page holds page_size tokens of every kv head.  Both kernels here and
// the attention kernels address it in 16-byte packets of E elements (8 fp16 or
// 16 fp8), laid out for the matrix-core operands that read them:
//     K [pages, kv_heads, head_dim / E, page_size, E]
//     V [pages, kv_heads, page_size / E, head_dim, E]
#include "device.h"

namespace spffn {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// Block tables.  With p tokens per page, request r of length len and add new
// tokens holds ceil(len / p) pages and needs ceil((len + add) / p) - held more,
// the off_r-th .. of the free list's end, off = exclusive sum of need; its
// tokens start at the exclusive sum of add.  A step has at most a few thousand
// requests, so every workgroup takes both sums for itself (a few KB from L2, no
// second launch and no workgroup waiting for another), keeps them in LDS, and
// then fills its share of the tokens' slots and of the new table entries; a
// token or a page finds its request by bisection of the sums.  The work is a
// handful of dependent loads: latency bounds it.
// ---------------------------------------------------------------------------
constexpr int kTabThreads = 256;

struct TabArgs {
    const int32_t *lens, *adds;
    int32_t *table;
    const int32_t *free_list, *n_free;
    int32_t *starts, *new_lens, *slots, *positions, *left;
    int R, width, free_cap, N, shift;  // shift: log2(page_size)
};

// Exclusive prefix of v over the workgroup's threads in order; *total the sum.
__device__ __forceinline__ int64_t block_scan64(int64_t v, int64_t *lds, int64_t *total) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    int64_t incl = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t u = __shfl_up(incl, o, 64);
        if (lane >= o) incl += u;
    }
    if (lane == 63) lds[wv] = incl;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kTabThreads / 64; ++w) {
        if (w < wv) before += lds[w];
        all += lds[w];
    }
    __syncthreads();
    *total = all;
    return before + incl - v;
}

__device__ __forceinline__ int clamp31(int64_t v) {
    return v > 0x7FFFFFFF ? 0x7FFFFFFF : (int)v;
}

// pages of a request: held and needed; false when it cannot be written at all
__device__ __forceinline__ bool tab_pages(const TabArgs &a, int len, int add, int &held, int &need) {
    held = need = 0;
    const int64_t p = (int64_t)1 << a.shift;
    if (len < 0 || add < 0 || (int64_t)len + add > (int64_t)a.width * p) return false;
    held = (int)(((int64_t)len + p - 1) >> a.shift);
    need = (int)(((int64_t)len + add + p - 1) >> a.shift) - held;
    return true;
}

// last index i in [0, n) with v[i] <= x (v ascending, v[0] <= x)
__device__ __forceinline__ int last_le(const int *v, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kTabThreads) void block_tables_kernel(TabArgs a) {
    extern __shared__ __align__(16) int tab_lds[];
    __shared__ int64_t scan[kTabThreads / 64];
    __shared__ int used_s, short_s;
    int *st = tab_lds;             // [R + 1] first token of each request
    int *off = tab_lds + a.R + 1;  // [R + 1] first new page of each request
    const int tid = threadIdx.x;
    int n_free = a.n_free[0];
    n_free = n_free < 0 ? 0 : n_free > a.free_cap ? a.free_cap : n_free;
    if (tid == 0) used_s = short_s = 0;

    int64_t tok_base = 0, page_base = 0;
    int used = 0, unserved = 0;
    for (int r0 = 0; r0 < a.R; r0 += kTabThreads) {
        const int r = r0 + tid;
        int len = 0, add = 0, held = 0, need = 0;
        bool fits = true;
        if (r < a.R) {
            len = a.lens[r];
            add = a.adds[r];
            fits = tab_pages(a, len, add, held, need);
        }
        int64_t tt, tp;
        const int64_t t0 = tok_base + block_scan64(add > 0 ? add : 0, scan, &tt);
        const int64_t p0 = page_base + block_scan64(need, scan, &tp);
        if (r < a.R) {
            st[r] = clamp31(t0);
            off[r] = clamp31(p0);
            const bool served = fits && (need == 0 || p0 + need <= n_free);
            if (p0 + need <= n_free) used = (int)(p0 + need);
            unserved += !served;
            if (blockIdx.x == 0) {
                a.starts[r] = clamp31(t0);
                a.new_lens[r] = served ? len + add : len;
            }
        }
        tok_base += tt;
        page_base += tp;
    }
    if (tid == 0) {
        st[a.R] = clamp31(tok_base);
        off[a.R] = clamp31(page_base);
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        if (used) atomicMax(&used_s, used);
        if (unserved) atomicAdd(&short_s, unserved);
        __syncthreads();
        if (tid == 0) {
            a.starts[a.R] = st[a.R];
            a.left[0] = n_free - used_s;
            a.left[1] = short_s;
        }
    }

    const int step = gridDim.x * kTabThreads;
    // new pages: the ones past the free list's end belong to unserved requests
    const int pages = off[a.R] < n_free ? off[a.R] : n_free;
    for (int j = blockIdx.x * kTabThreads + tid; j < pages; j += step) {
        const int r = last_le(off, a.R, j);
        int held, need;
        tab_pages(a, a.lens[r], a.adds[r], held, need);
        if ((int64_t)off[r] + need <= n_free)
            a.table[(size_t)r * a.width + held + (j - off[r])] = a.free_list[n_free - 1 - j];
    }
    for (int64_t n = (int64_t)blockIdx.x * kTabThreads + tid; n < a.N; n += step) {
        int slot = -1, pos = -1;
        if (n < st[a.R]) {
            const int r = last_le(st, a.R, (int)n);
            const int len = a.lens[r], add = a.adds[r];
            int held, need;
            const bool fits = tab_pages(a, len, add, held, need);
            // a negative length has no positions; any other keeps them, served or not
            const int64_t at = (int64_t)len + (n - st[r]);
            pos = len < 0 ? -1 : clamp31(at);
            if (fits && (need == 0 || (int64_t)off[r] + need <= n_free)) {
                const int b = (int)(at >> a.shift);
                const int e = b < held ? a.table[(size_t)r * a.width + b]
                                       : a.free_list[n_free - 1 - (off[r] + b - held)];
                if (e >= 0) slot = (e << a.shift) | (int)(at & ((1 << a.shift) - 1));
            }
        }
        a.slots[n] = slot;
        a.positions[n] = pos;
    }
}

hipError_t launch_block_tables(const int32_t *lens, const int32_t *adds, int R, int shift,
                               int32_t *table, int width, const int32_t *free_list, int free_cap,
                               const int32_t *n_free, int32_t *starts, int32_t *new_lens,
                               int32_t *slots, int32_t *positions, int N, int32_t *left,
                               hipStream_t s) {
    TabArgs a{lens, adds, table, free_list, n_free, starts, new_lens,
              slots, positions, left, R, width, free_cap, N, shift};
    const int64_t most = (int64_t)N > (int64_t)R ? N : R;
    int64_t wgs = (most + kTabThreads - 1) / kTabThreads;
    wgs = wgs < 1 ? 1 : wgs > 512 ? 512 : wgs;
    block_tables_kernel<<<(int)wgs, kTabThreads, (size_t)(a.R + 1) * 8, s>>>(a);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Append.  Each workgroup takes T (16 or 64) tokens of one head, keys or values.
//   keys:   rows are read along the dimensions, rounded into LDS and stored from
//           there a packet (E dimensions of a token) per thread, tokens fastest:
//           neighbouring slots write neighbouring packets, so that both sides
//           move whole cache lines;
//   values: a packet is E neighbouring slots of one dimension.  Where E tokens of
//           the input run through a whole packet, the workgroup that has the
//           first of them writes it, a thread per dimension and one 16-byte
//           store; the tokens of broken packets (a decode step's are, most of
//           them) are stored element by element.
// HBM bounds long inputs (each element is read once and written once), the
// launch short ones.  The conversion is one rounding: fp16 to nearest, fp8 the
// nearest E4M3 value of x / scale (an fp32 division), saturating at +-448 (NaN
// stays NaN).
// ---------------------------------------------------------------------------
struct AppArgs {
    const void *k, *v;
    uint8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *slots;
    int64_t ldk, ldv;
    int N, H, shift;
    int64_t n_slots;
};

// x / s, correctly rounded, for one s and many x: with y the rounded reciprocal,
// q = x y is within two steps, and each q + (x - q s) y, the rest taken exactly,
// comes within the last rounding.  Quotients past E4M3's range need no more than
// their size.  Scales so small or large that y or the rest leaves the normal
// range are divided by as they are.
struct Quotient {
    float s, y;
    bool plain;
    __device__ __forceinline__ explicit Quotient(float scale) : s(scale), y(1.0f / scale) {
        plain = !(fabsf(scale) > 1e-18f && fabsf(scale) < 1e18f);
    }
    __device__ __forceinline__ float operator()(float x) const {
        if (plain) return x / s;
        float q = x * y;
        const float q1 = fmaf(fmaf(-q, s, x), y, q);
        const float q2 = fmaf(fmaf(-q1, s, x), y, q1);
        return fabsf(q) < 1024.0f ? q2 : q;  // (infinities and NaN too)
    }
};

// Four values as E4M3, saturating; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const float sum = (a + b) + (c + d);
    if (!(fabsf(sum) < __builtin_inff())) {  // rare: some value may be NaN
        a = a > 448.0f ? 448.0f : a < -448.0f ? -448.0f : a;
        b = b > 448.0f ? 448.0f : b < -448.0f ? -448.0f : b;
        c = c > 448.0f ? 448.0f : c < -448.0f ? -448.0f : c;
        d = d > 448.0f ? 448.0f : d < -448.0f ? -448.0f : d;
    } else {
        a = __builtin_amdgcn_fmed3f(a, -448.0f, 448.0f);
        b = __builtin_amdgcn_fmed3f(b, -448.0f, 448.0f);
        c = __builtin_amdgcn_fmed3f(c, -448.0f, 448.0f);
        d = __builtin_amdgcn_fmed3f(d, -448.0f, 448.0f);
    }
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// E fp32 values as one packet.
template <bool FP8>
__device__ __forceinline__ uint4 to_packet(const float *v) {
    if constexpr (FP8) {
        return make_uint4(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]),
                          e4m3x4(v[8], v[9], v[10], v[11]), e4m3x4(v[12], v[13], v[14], v[15]));
    } else {
        half8 h;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = (_Float16)v[e];
        return __builtin_bit_cast(uint4, h);
    }
}

// Four source elements from p on, as fp32.
template <bool SRC16>
__device__ __forceinline__ float4 four(const void *base, size_t at) {
    if constexpr (SRC16) {
        typedef _Float16 half4 __attribute__((ext_vector_type(4)));
        const half4 x = *reinterpret_cast<const half4 *>(static_cast<const _Float16 *>(base) + at);
        return make_float4((float)x[0], (float)x[1], (float)x[2], (float)x[3]);
    } else {
        return *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
    }
}

template <bool FP8, bool SRC16, int D, int T>
__global__ __launch_bounds__(256) void kv_append_kernel(AppArgs a) {
    constexpr int E = FP8 ? 16 : 8, ES = FP8 ? 1 : 2;
    typedef typename std::conditional<SRC16, _Float16, float>::type S;
    const int n0 = blockIdx.x * T, h = blockIdx.y, tid = threadIdx.x;
    const int ps = 1 << a.shift;
    auto slot_of = [&](int n) {
        const int s = n >= 0 && n < a.N ? a.slots[n] : -1;
        return s < a.n_slots ? s : -1;
    };
    if (blockIdx.z == 0) {
        constexpr int pitch = D * ES + 16, Q = D / 4, PER = (T * Q + 255) / 256, npk = D / E;
        __shared__ __align__(16) uint8_t tile[T * pitch];
        const int t = tid % T, slot = slot_of(n0 + t);
        float4 x[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = tid + 256 * k, n = n0 + i / Q;
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < T * Q && n < a.N)
                x[k] = four<SRC16>(a.k, (size_t)n * a.ldk + (size_t)h * D + 4 * (i % Q));
        }
        const Quotient by(FP8 ? a.ks[h] : 1.0f);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = tid + 256 * k;
            uint8_t *to = tile + i / Q * pitch + 4 * (i % Q) * ES;
            if (i >= T * Q) break;
            if constexpr (FP8) {
                *reinterpret_cast<uint32_t *>(to) = e4m3x4(by(x[k].x), by(x[k].y), by(x[k].z), by(x[k].w));
            } else {
                typedef _Float16 half4 __attribute__((ext_vector_type(4)));
                *reinterpret_cast<half4 *>(to) = half4{(_Float16)x[k].x, (_Float16)x[k].y,
                                                       (_Float16)x[k].z, (_Float16)x[k].w};
            }
        }
        __syncthreads();
        if (slot < 0) return;
        const size_t page = (size_t)(slot >> a.shift), o = (size_t)(slot & (ps - 1));
        uint4 *dst = reinterpret_cast<uint4 *>(a.kc) + (page * a.H + h) * npk * ps + o;
        for (int pk = tid / T; pk < npk; pk += 256 / T)
            dst[(size_t)pk * ps] = *reinterpret_cast<const uint4 *>(tile + t * pitch + pk * 16);
        return;
    }
    // slots from E - 1 before the first token on (a packet may have begun there)
    __shared__ int near[T + 2 * (E - 1)];
    __shared__ uint64_t whole_s, lead_s;
    for (int i = tid; i < T + 2 * (E - 1); i += 256) near[i] = slot_of(n0 - (E - 1) + i);
    __syncthreads();
    if (tid < 64) {  // which tokens belong to a whole packet, and which begin one
        bool all = false, lead = false;
        if (tid < T) {
            const int slot = near[tid + E - 1], o = slot & (E - 1);
            all = slot >= 0;
#pragma unroll
            for (int e = 0; e < E; ++e) all = all && near[(tid + E - 1) - o + e] == slot - o + e;
            lead = all && o == 0;
        }
        const uint64_t w = __ballot(all), l = __ballot(lead);
        if (tid == 0) {
            whole_s = w;
            lead_s = l;
        }
    }
    __syncthreads();
    const uint64_t whole = whole_s, leads = lead_s;
    const int n_lead = __popcll(leads);
    const Quotient by(FP8 ? a.vs[h] : 1.0f);
    const S *src = static_cast<const S *>(a.v) + (size_t)h * D;
    auto packet_at = [&](int slot, int d) {  // bytes
        const size_t row = ((size_t)(slot >> a.shift) * a.H + h) * (size_t)(ps / E) + ((slot & (ps - 1)) / E);
        return a.vc + (row * D + d) * 16;
    };
    if (n_lead) {
        constexpr int PER = (T / E * D + 255) / 256;  // packets of a thread: whole ones are E apart
        float v[PER][E];
        int slot[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = tid + 256 * k, p = i / D, d = i % D;
            slot[k] = -1;
            if (p >= n_lead) continue;
            uint64_t m = leads;
            for (int x = 0; x < p; ++x) m &= m - 1;
            const int t = __ffsll((long long)m) - 1;
            slot[k] = near[t + E - 1];
            const S *from = src + (size_t)(n0 + t) * a.ldv + d;
#pragma unroll
            for (int e = 0; e < E; ++e) v[k][e] = (float)from[(size_t)e * a.ldv];
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (slot[k] < 0) continue;
            if (FP8) {
#pragma unroll
                for (int e = 0; e < E; ++e) v[k][e] = by(v[k][e]);
            }
            *reinterpret_cast<uint4 *>(packet_at(slot[k], (tid + 256 * k) % D)) = to_packet<FP8>(v[k]);
        }
    }
    // the other tokens, by elements
    if (whole == ~0ull >> (64 - T)) return;
#pragma unroll 4
    for (int i = tid; i < T * D; i += 256) {
        const int t = i / D, d = i % D, slot = near[t + E - 1];
        if (slot < 0 || ((whole >> t) & 1)) continue;
        const float v = (float)src[(size_t)(n0 + t) * a.ldv + d];
        uint8_t *dst = packet_at(slot, d) + (slot & (E - 1)) * ES;
        if constexpr (FP8) *dst = (uint8_t)e4m3x4(by(v), 0.0f, 0.0f, 0.0f);
        else *reinterpret_cast<_Float16 *>(dst) = (_Float16)v;
    }
}

template <int D, int T>
hipError_t launch_append_dim(const KvCache &c, const AppArgs &a, bool src16, hipStream_t s) {
    const dim3 grid((a.N - 1) / T + 1, c.H, 2);
    if (c.fp8) {
        if (src16) kv_append_kernel<true, true, D, T><<<grid, 256, 0, s>>>(a);
        else kv_append_kernel<true, false, D, T><<<grid, 256, 0, s>>>(a);
    } else {
        if (src16) kv_append_kernel<false, true, D, T><<<grid, 256, 0, s>>>(a);
        else kv_append_kernel<false, false, D, T><<<grid, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <int T>
hipError_t launch_append(const KvCache &c, const AppArgs &a, bool src16, hipStream_t s) {
    switch (c.D) {
        case 64: return launch_append_dim<64, T>(c, a, src16, s);
        case 96: return launch_append_dim<96, T>(c, a, src16, s);
        case 128: return launch_append_dim<128, T>(c, a, src16, s);
        default: return launch_append_dim<256, T>(c, a, src16, s);
    }
}

hipError_t launch_kv_append(const KvCache &c, const void *k, const void *v, bool src16, int64_t ldk,
                            int64_t ldv, const int32_t *slots, int N, hipStream_t s) {
    const AppArgs a{k, v, c.k, c.v, c.ks, c.vs, slots, ldk, ldv, N, c.H, c.shift,
                    (int64_t)c.pages << c.shift};
    // A workgroup is a chain of waits (slots, rows, stores) whatever it moves, so it moves as
    // much as fits its registers once the chip is full of them (8191 tokens of 8 heads to fp8,
    // 84 MB: 24 us, with 16 tokens a workgroup 38 us); a step's few tokens spread over more.
    const bool many = (int64_t)N * c.H * 2 >= (int64_t)64 * 512;
    return many ? launch_append<64>(c, a, src16, s) : launch_append<16>(c, a, src16, s);
}

}  // namespace spffn
