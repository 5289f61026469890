// Matrix-vector products with 4-bit weights and group scales, 1..16 tokens:
//
//     y[b, i] = r_b * sum_c (q[i, c] - z[i, c / G]) s[i, c / G] x[b, c]
//               + bias[i] + resid[b, i],   r_b = 1 or 1 / sqrt(mean_c x[b, c]^2 + eps)
//
// Every code is read once, so HBM bounds the product; what has to stay out of
// the way is the widening of the codes and the 16 multiply-adds per code.  The
// products run on v_mfma_f32_16x16x32_f16 for every batch, one token included:
//
//   * weights are the A operand.  q - z is a small integer, exact in binary16:
//     a nibble under the exponent of 1024 reads as 1024 + q (or 1024 + 16 q), and
//     one packed operation takes 1024 + z off (or divides by 16 and takes 64 + z
//     off), so eight codes cost nine instructions.  (Leaving the constant in and
//     taking its share of the sum off at the end would save two of them, and q as
//     a subnormal half four; the first loses what a large activation times 16 + q
//     rounds away where its weight is 0, the second a relative 7e-5, since the
//     product of a subnormal drops low bits.)  The scale is applied in fp32 to a
//     group's sum, so no weight is ever rounded;
//   * activations are the B operand, hi + lo halves of x scaled by a power of
//     two (largest magnitude in [2^14, 2^15)): about 22 significant bits down to
//     2^-18 of the largest, an absolute 2^-40 of it below.  For B <= 8 the hi
//     halves are columns 0..7 and the lo halves columns 8..15 of one instruction,
//     for B > 8 they take one each into the same accumulator;
//   * B <= 2 is one launch: a wave owns whole blocks of 128 columns (wave, wave +
//     W, ...) of a tile of 16 rows and splits their activations itself, with a
//     scale per token and block; no wave waits for another before the final sum,
//     which is taken in a fixed order;
//   * B > 2 splits the activations in a launch of its own, and the product reads
//     the halves from L2.  (Sharing them through LDS between waves of different
//     rows, a barrier every two or four blocks, was slower: 9216 x 8192 and five
//     tokens 22.9 us against 20.3, 36864 x 12288 and sixteen 78.7 against 72.)
//     The RMS norm needs no pass of its own in either: it has no gain, so it is
//     one factor per token at the end.
//
// Measured in a replayed graph: 4096 x 4096, one token 5.4 us (9.5 MB, mostly the
// launch and one chain of loads); 10240 x 8192, one token 16.6 us (44 MB, 2.65
// TB/s); 9216 x 8192, five tokens 20.3 us; 36864 x 12288, sixteen tokens 72 to 77
// us (244 MB, 3.3 TB/s).  A plain read of as many bytes reaches 7 TB/s: between
// the two stand the waits of each wave for its own codes, since a block's work is
// short (a deeper prefetch costs more waves than it saves).
//
// Packed layout (launch_q4_pack): per tile of 16 rows and block of 128 columns
// 1 KiB of codes in the order of one wave's 16-byte loads -- lane l = 16 g + m
// holds row m, word w the eight columns 32 w + 8 g + e, code 2i in nibble i and
// code 2i + 1 in nibble i + 4 -- then all scales [tile, block, row, group] fp16,
// then all zero points (same shape, bytes): a lane's are one load each.  Rows and columns are padded with
// zero codes and zero scales.
#include "device.h"

namespace spffn {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

namespace {

constexpr int kBlk = 128;         // columns per block
constexpr int kRow = 16;          // rows per tile
constexpr int kXPitch = 136;      // halves per token and plane in LDS (128 + 16 bytes of padding)

__device__ __forceinline__ uint32_t regroup(uint32_t s) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w |= ((s >> (8 * i)) & 15u) << (4 * i);
        w |= ((s >> (8 * i + 4)) & 15u) << (16 + 4 * i);
    }
    return w;
}

// One thread per 16-byte packet; scales and zero points by the first threads
// of each block of 64.
__global__ __launch_bounds__(256) void q4_pack_kernel(const uint8_t *__restrict__ codes,
                                                      const uint16_t *__restrict__ scales,
                                                      const uint8_t *__restrict__ zeros, int rows,
                                                      int cols, int group, int kb_n, int64_t n_rec,
                                                      uint8_t *__restrict__ packed) {
    const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t rec = t >> 6;
    if (rec >= n_rec) return;
    const int lane = (int)(t & 63), m = lane & 15, g = lane >> 4;
    const int rt = (int)(rec / kb_n), kb = (int)(rec - (int64_t)rt * kb_n);
    const int row = rt * kRow + m;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = kb * kBlk + 32 * i + 8 * g;  // cols % 32 == 0: eight columns or none
        uint32_t s = 0;
        if (row < rows && col < cols) {
            const uint8_t *p = codes + (size_t)row * (cols / 2) + col / 2;
            s = (uint32_t)p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16 | (uint32_t)p[3] << 24;
        }
        w[i] = regroup(s);
    }
    *reinterpret_cast<uint4 *>(packed + (size_t)t * 16) = make_uint4(w[0], w[1], w[2], w[3]);

    const int ng = kBlk / group, groups = (cols + group - 1) / group;
    if (lane < 16 * ng) {
        const int gi = lane >> 4, gg = kb * ng + gi;
        const bool in = row < rows && gg < groups;
        uint16_t *sc = reinterpret_cast<uint16_t *>(packed + (size_t)n_rec * 1024);
        const size_t at = ((size_t)rec * 16 + m) * ng + gi;
        sc[at] = in ? scales[(size_t)row * groups + gg] : (uint16_t)0;
        if (zeros)
            packed[(size_t)n_rec * (1024 + 32 * ng) + at] =
                in ? (uint8_t)(zeros[(size_t)row * groups + gg] & 15) : (uint8_t)0;
    }
}

struct Q4Args {
    const uint8_t *packed;
    const float *x, *bias, *resid;
    float *y;
    int rows, cols, kb_n, B;
    int64_t n_rec;
    float eps;  // < 0: no normalisation
};

// The masks of the codes' bits and the exponent of 1024, in registers whose
// values the compiler does not see: it then makes one and-or of each use, not two
// instructions with a literal each.
struct CodeBits {
    uint32_t low, high, exponent;
    __device__ __forceinline__ CodeBits() : low(0x000F000Fu), high(0x00F000F0u), exponent(0x64006400u) {
        asm("" : "+s"(low));
        asm("" : "+s"(high));
        asm("" : "+v"(exponent));
    }
    __device__ __forceinline__ half2v operator()(uint32_t w, uint32_t mask) const {
        return __builtin_bit_cast(half2v, (w & mask) | exponent);
    }
};

// What a zero point takes off 1024 + q, and off 64 + q.
struct Offsets {
    half2v one, sixteen;
    template <bool ZP>
    __device__ __forceinline__ static Offsets of(uint32_t z) {
        const _Float16 zp = ZP ? (_Float16)(float)(z & 15u) : (_Float16)8.0f;
        const _Float16 a = (_Float16)-1024.0f - zp, b = (_Float16)-64.0f - zp;
        return Offsets{half2v{a, a}, half2v{b, b}};
    }
};

// A lane needs the scales of rows 4g .. 4g + 3 of a record, as every lane of its
// row of 16 does.  It loads those of one, 4g + n % 4, and takes the others from
// the lanes of its quad: a quarter of the bytes through the load path, where
// whole loads of the same four rows by every lane cost as much as the codes.
template <int NG>
struct Scales {
    static constexpr int DW = NG < 2 ? 1 : NG / 2;
    uint32_t own[DW];
    __device__ __forceinline__ void load(const uint8_t *p) {
        if constexpr (NG == 1) own[0] = *reinterpret_cast<const uint16_t *>(p);
        else if constexpr (NG == 2) own[0] = *reinterpret_cast<const uint32_t *>(p);
        else {
            const uint2 x = *reinterpret_cast<const uint2 *>(p);
            own[0] = x.x;
            own[1] = x.y;
        }
    }
    template <int ROW>
    __device__ __forceinline__ half2v quad(int dw) const {  // row 4g + ROW, groups 2 dw, 2 dw + 1
        return __builtin_bit_cast(half2v, __builtin_amdgcn_mov_dpp((int)own[dw], ROW * 0x55, 0xF, 0xF, true));
    }
    __device__ __forceinline__ _Float16 operator()(int row, int group) const {
        const int dw = group / 2;
        const half2v x = row == 0 ? quad<0>(dw) : row == 1 ? quad<1>(dw) : row == 2 ? quad<2>(dw)
                                                                                    : quad<3>(dw);
        return x[group % 2];
    }
};

// The NG zero points of a row, a byte each.
template <int NG>
__device__ __forceinline__ uint32_t load_zeros(const uint8_t *p) {
    if constexpr (NG == 1) return *p;
    else if constexpr (NG == 2) return *reinterpret_cast<const uint16_t *>(p);
    else return *reinterpret_cast<const uint32_t *>(p);
}

// Eight codes as q - z.
__device__ __forceinline__ half8 widen(uint32_t w, const CodeBits &bits, const Offsets &off) {
    const half2v sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t h = w >> 8;
    const half2v a = bits(w, bits.low) + off.one;
    const half2v b = __builtin_elementwise_fma(bits(w, bits.high), sixteenth, off.sixteen);
    const half2v c = bits(h, bits.low) + off.one;
    const half2v d = __builtin_elementwise_fma(bits(h, bits.high), sixteenth, off.sixteen);
    return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Magnitudes are compared as integers: one instruction each (a float maximum
// would first quiet NaNs), and whatever is not finite sorts above the rest.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
    return v > o ? v : o;
}

// The largest value of each group of LPT (16, 32 or 64) lanes, in every lane of it.
template <int LPT>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    v = dpp_max<0xB1>(v);   // quad_perm [1,0,3,2]
    v = dpp_max<0x4E>(v);   // quad_perm [2,3,0,1]
    v = dpp_max<0x141>(v);  // row_half_mirror
    v = dpp_max<0x140>(v);  // row_mirror
    if constexpr (LPT == 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = r[0] > r[1] ? r[0] : r[1];
    }
    if constexpr (LPT == 64) {
        const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
        const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
        const uint32_t x = a > b ? a : b, y = c > d ? c : d;
        v = x > y ? x : y;  // one value for the wave, in a scalar register
    }
    return v;
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }


constexpr uint32_t kInf = 0x7F800000u;

// Scale that puts a largest magnitude m in [2^14, 2^15), and its inverse.
__device__ __forceinline__ uint32_t scale_bits(uint32_t m) {
    const uint32_t eb = m >> 23;
    return eb < 16 ? 16 : eb;
}
__device__ __forceinline__ float scale_up(uint32_t eb) { return __uint_as_float((268u - eb) << 23); }
__device__ __forceinline__ float scale_down(uint32_t eb) { return __uint_as_float((eb - 14u) << 23); }

// hi and lo halves of v * up; an infinity or NaN has lo 0 (not inf - inf).
__device__ __forceinline__ void split(float v, float up, bool odd, _Float16 &hi, _Float16 &lo) {
    hi = (_Float16)(v * up);
    lo = (_Float16)fmaf(v, up, -(float)hi);
    if (odd && magnitude(v) >= kInf) lo = (_Float16)0.0f;
}

// Fixed-order sum over the workgroup's waves of one output: red [W][RT][16][16]
// holds a wave's sums per column and row; TWO adds the lo halves' column b + 8.
template <int RT, int W, bool TWO>
__device__ __forceinline__ float sum_waves(const float *red, int b, int t, int r) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        v += red[((w * RT + t) * 16 + b) * 16 + r];
        if (TWO) v += red[((w * RT + t) * 16 + b + 8) * 16 + r];
    }
    return v;
}

// ---------------------------------------------------------------------------
// B <= 2: one launch.  A wave owns blocks wv, wv + W, ... of RT tiles, with the
// codes of DW of them in flight, and splits those blocks' activations itself, XB
// blocks at a time (a scale per token and block), through LDS of its own.
// ---------------------------------------------------------------------------
template <int NG, bool ZP, int B, int RT, int W, int DW>
__global__ __launch_bounds__(64 * W, 4) void q4mv_kernel(Q4Args a) {
    constexpr int E = 2 * B;                  // activations per lane and block
    constexpr int XB = 4 / B;
    constexpr int LPT = kBlk / E;             // lanes per token
    constexpr int SPG = 4 / NG;               // instructions per group
    constexpr int U = XB > DW ? XB : DW;
    constexpr int AREA = 2 * B * kXPitch + 32;  // halves: hi and lo planes, factors
    constexpr size_t STAGE = (size_t)W * XB * AREA * 2;
    constexpr size_t RED = (size_t)W * RT * 1024 + (size_t)W * 64;
    __shared__ __align__(16) uint8_t smem[STAGE > RED ? STAGE : RED];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int rt0 = blockIdx.x * RT;
    const int n_rt = (a.rows + kRow - 1) / kRow;
    _Float16 *xs = reinterpret_cast<_Float16 *>(smem) + wv * XB * AREA;

    const uint8_t *sc_base = a.packed + (size_t)a.n_rec * 1024;
    const uint8_t *zp_base = sc_base + (size_t)a.n_rec * 32 * NG;

    size_t rec0[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int rt = rt0 + t < n_rt ? rt0 + t : n_rt - 1;  // a tile past the end is not stored
        rec0[t] = (size_t)rt * a.kb_n;
    }

    const int tok = lane / LPT, el = (lane % LPT) * E;  // this lane's token, its first column
    const int col_tok = (n & 7) < B ? (n & 7) : B - 1;
    const int b_at = (n >= 8 ? B * kXPitch : 0) + col_tok * kXPitch + 8 * g;

    const CodeBits bits;
    f32x4 acc[RT];
    float ss = 0.0f;
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};

    uint4 cw[DW][RT];
    Scales<NG> cs[DW][RT];
    uint32_t cz[DW][RT];
    float cx[XB][E];
    auto load_w = [&](int st, int kb) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const size_t rec = rec0[t] + kb;
            cw[st][t] = __builtin_bit_cast(
                uint4, __builtin_nontemporal_load(
                           reinterpret_cast<const u32x4_t *>(a.packed + rec * 1024) + lane));
            cs[st][t].load(sc_base + (rec * 16 + 4 * g + (n & 3)) * (2 * NG));
            if (ZP) cz[st][t] = load_zeros<NG>(zp_base + (rec * 16 + n) * NG);
        }
    };
    auto load_x = [&](int xb, int kb) {
        const int c = kb * kBlk + el;
        const bool in = c < a.cols;  // cols % 32 == 0: all E columns or none
        const float *src = a.x + (size_t)tok * a.cols + (in ? c : 0);
        if constexpr (E == 2) {
            const float2 v = *reinterpret_cast<const float2 *>(src);
            cx[xb][0] = in ? v.x : 0.0f;
            cx[xb][1] = in ? v.y : 0.0f;
        } else {
            const float4 v = *reinterpret_cast<const float4 *>(src);
            cx[xb][0] = in ? v.x : 0.0f;
            cx[xb][1] = in ? v.y : 0.0f;
            cx[xb][2] = in ? v.z : 0.0f;
            cx[xb][3] = in ? v.w : 0.0f;
        }
    };

#pragma unroll
    for (int b = 0; b < XB; ++b)
        if (wv + b * W < a.kb_n) load_x(b, wv + b * W);
#pragma unroll
    for (int d = 0; d < DW; ++d)
        if (wv + d * W < a.kb_n) load_w(d, wv + d * W);

    // U blocks from kb0 on.  ALL: they and the DW after them are all there, so no load hangs
    // on a condition (one that may be skipped would make the ones behind it be waited for as
    // if it had been).
    auto blocks = [&](auto all, int kb0) {
        constexpr bool ALL = decltype(all)::value;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = kb0 + u * W;
            if (!ALL && kb >= a.kb_n) break;
            if (u % XB == 0) {
                // ---- split the next XB blocks of activations ----
                uint32_t m[XB], top = 0;
#pragma unroll
                for (int b = 0; b < XB; ++b) {
                    if (!ALL && b > 0 && kb + b * W >= a.kb_n) {
#pragma unroll
                        for (int e = 0; e < E; ++e) cx[b][e] = 0.0f;
                    }
                    uint32_t v = 0;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const uint32_t q = magnitude(cx[b][e]);
                        v = v > q ? v : q;
                    }
                    if (a.eps >= 0.0f) {
#pragma unroll
                        for (int e = 0; e < E; ++e) ss = fmaf(cx[b][e], cx[b][e], ss);
                    }
                    m[b] = lanes_max<LPT>(v);
                    top = top > m[b] ? top : m[b];
                }
                const bool odd = __any(top >= kInf);
                if (odd) {
                    // an infinity or NaN: scale by the finite values
#pragma unroll
                    for (int b = 0; b < XB; ++b) {
                        uint32_t v = 0;
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const uint32_t q = magnitude(cx[b][e]);
                            v = q < kInf && q > v ? q : v;
                        }
                        m[b] = lanes_max<LPT>(v);
                    }
                }
                __builtin_amdgcn_wave_barrier();  // the blocks before have been read
#pragma unroll
                for (int b = 0; b < XB; ++b) {
                    _Float16 *xh = xs + b * AREA, *xl = xh + B * kXPitch;
                    const uint32_t eb = scale_bits(m[b]);
                    const float up = scale_up(eb);
                    _Float16 hi[E], lo[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) split(cx[b][e], up, odd, hi[e], lo[e]);
                    if constexpr (E == 2) {
                        *reinterpret_cast<half2v *>(xh + tok * kXPitch + el) = half2v{hi[0], hi[1]};
                        *reinterpret_cast<half2v *>(xl + tok * kXPitch + el) = half2v{lo[0], lo[1]};
                    } else {
                        *reinterpret_cast<half4 *>(xh + tok * kXPitch + el) =
                            half4{hi[0], hi[1], hi[2], hi[3]};
                        *reinterpret_cast<half4 *>(xl + tok * kXPitch + el) =
                            half4{lo[0], lo[1], lo[2], lo[3]};
                    }
                    if (el == 0) reinterpret_cast<float *>(xl + B * kXPitch)[tok] = scale_down(eb);
                }
#pragma unroll
                for (int b = 0; b < XB; ++b) {
                    const int kx = kb + (XB + b) * W;
                    if (ALL) load_x(b, kx < a.kb_n ? kx : kb);
                    else if (kx < a.kb_n) load_x(b, kx);
                }
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            }
            const _Float16 *xh = xs + (u % XB) * AREA;
            half8 bx[4];
#pragma unroll
            for (int w = 0; w < 4; ++w)
                bx[w] = *reinterpret_cast<const half8 *>(xh + b_at + 32 * w);
            const float f = reinterpret_cast<const float *>(xh + 2 * B * kXPitch)[col_tok];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const uint4 q = cw[u % DW][t];
                const uint32_t words[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    const Offsets off = Offsets::of<ZP>(cz[u % DW][t] >> (8 * i));
                    f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int w = i * SPG; w < (i + 1) * SPG; ++w)
                        z = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(words[w], bits, off), bx[w], z,
                                                                   0, 0, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[t][j] = fmaf(z[j], fmaf((float)cs[u % DW][t](j, i), f, 0.0f), acc[t][j]);
                }
            }
            if (ALL || kb + DW * W < a.kb_n) load_w(u % DW, kb + DW * W);
        }
    };
    int kb0 = wv;
    for (; kb0 + (U + DW - 1) * W < a.kb_n; kb0 += U * W) blocks(std::true_type{}, kb0);
    for (; kb0 < a.kb_n; kb0 += U * W) blocks(std::false_type{}, kb0);

    // ---- fixed-order sum over the workgroup's waves, scale, bias, residual ----
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);            // [W][RT][16 columns][16 rows]
    float *sq = red + W * RT * 256;                          // [W][16] sums of squares
#pragma unroll
    for (int t = 0; t < RT; ++t)
        *reinterpret_cast<f32x4 *>(red + ((wv * RT + t) * 16 + n) * 16 + 4 * g) = acc[t];
    if (a.eps >= 0.0f) {
#pragma unroll
        for (int o = 1; o < LPT; o <<= 1) ss += __shfl_xor(ss, o, 64);
        if (el == 0) sq[wv * 16 + tok] = ss;
    }
    __syncthreads();
    for (int o = tid; o < RT * kRow * B; o += 64 * W) {
        const int b = o / (RT * kRow), lr = o - b * (RT * kRow);
        const int row = rt0 * kRow + lr;
        if (row >= a.rows) continue;
        float v = sum_waves<RT, W, true>(red, b, lr >> 4, lr & 15);
        if (a.eps >= 0.0f) {
            float q = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) q += sq[w * 16 + b];
            v *= 1.0f / sqrtf(q / (float)a.cols + a.eps);
        }
        if (a.bias) v += a.bias[row];
        const size_t at = (size_t)b * a.rows + row;
        if (a.resid) v += a.resid[at];
        a.y[at] = v;
    }
}

// ---------------------------------------------------------------------------
// B > 2: splitting the activations costs a wave more than the codes of one tile
// do (16 tokens: 160 instructions a block against 50), so a first launch does it
// once, one workgroup per token: the row's largest magnitude gives the token's
// scale, the halves go to the workspace in the order of the B operand -- block,
// instruction, [hi, lo for B > 8], lane, 16 bytes -- and the factor that undoes
// the scale, with the RMS norm in it, behind them.
// ---------------------------------------------------------------------------
constexpr int kSplitThreads = 1024;

struct SplitArgs {
    const float *x;
    _Float16 *xp;
    float *fac;
    int cols, kb_n, wide;
    float eps;
    int *done;
    int n_done;  // counters of the product's launch, to be cleared
};

__global__ __launch_bounds__(kSplitThreads) void q4_split_kernel(SplitArgs a) {
    __shared__ uint32_t mx[kSplitThreads / 64];
    __shared__ float sq[kSplitThreads / 64];
    const int tok = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const float *x = a.x + (size_t)tok * a.cols;
    for (int i = tok * kSplitThreads + tid; i < a.n_done; i += gridDim.x * kSplitThreads) a.done[i] = 0;
    constexpr int KEEP = 2;  // packets of 8 a thread keeps (16384 columns), the rest is read twice
    float keep[KEEP][8];
    uint32_t m = 0;
    bool odd = false;
    float ss = 0.0f;
    const int n_pk = a.cols / 8;
    int i = 0;
    for (int p = tid; p < n_pk; p += kSplitThreads, ++i) {
        const float4 u = reinterpret_cast<const float4 *>(x)[2 * p];
        const float4 v = reinterpret_cast<const float4 *>(x)[2 * p + 1];
        const float e[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t q = magnitude(e[k]);
            odd = odd || q >= kInf;
            m = q < kInf && q > m ? q : m;
            ss = fmaf(e[k], e[k], ss);
        }
#pragma unroll
        for (int s = 0; s < KEEP; ++s)
            if (s == i) {
#pragma unroll
                for (int k = 0; k < 8; ++k) keep[s][k] = e[k];
            }
    }
    m = lanes_max<64>(m);
    ss = wave_sum(ss);
    if (lane == 0) {
        mx[wv] = m;
        sq[wv] = ss;
    }
    __syncthreads();
    ss = 0.0f;
#pragma unroll
    for (int w = 0; w < kSplitThreads / 64; ++w) {
        m = mx[w] > m ? mx[w] : m;
        ss += sq[w];
    }
    const uint32_t eb = scale_bits(m);
    const float up = scale_up(eb);
    if (tid == 0) {
        const float r = a.eps >= 0.0f ? 1.0f / sqrtf(ss / (float)a.cols + a.eps) : 1.0f;
        a.fac[2 * tok] = scale_down(eb);
        a.fac[2 * tok + 1] = r;
    }
    i = 0;
    // columns past cols (the last block's end) are zeros
    for (int p = tid; p < a.kb_n * (kBlk / 8); p += kSplitThreads, ++i) {
        float e[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (i < KEEP && p < n_pk) {
#pragma unroll
            for (int s = 0; s < KEEP; ++s)
                if (s == i) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) e[k] = keep[s][k];
                }
        } else if (p < n_pk) {
            const float4 u = reinterpret_cast<const float4 *>(x)[2 * p];
            const float4 v = reinterpret_cast<const float4 *>(x)[2 * p + 1];
            e[0] = u.x; e[1] = u.y; e[2] = u.z; e[3] = u.w;
            e[4] = v.x; e[5] = v.y; e[6] = v.z; e[7] = v.w;
        }
        half8 hi, lo;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            _Float16 h, l;
            split(e[k], up, odd, h, l);
            hi[k] = h;
            lo[k] = l;
        }
        // packet p holds columns 8p ..: instruction p / 4 (of 32 columns), lane group p % 4
        const size_t at = (size_t)(p >> 2) * (a.wide ? 128 : 64) + (p & 3) * 16 + tok;
        reinterpret_cast<half8 *>(a.xp)[at] = hi;
        reinterpret_cast<half8 *>(a.xp)[at + (a.wide ? 64 : 8)] = lo;
    }
}

// The product itself: as q4mv_kernel, with the B operand loaded as it is (from
// L2: every workgroup reads it, once per RT tiles) and one scale per token, so
// that a group's scale is one mixed-precision multiply-add per output.
struct MmArgs {
    Q4Args q;
    const _Float16 *xp;
    const float *fac;
    float *part;  // [row groups][KS][B][rows]
    int *done;    // [row groups] workgroups counted, 0 before the launch
};

template <int NG, bool ZP, bool WIDE, int RT, int W, int DW>
__global__ __launch_bounds__(64 * W, 4) void q4mm_kernel(MmArgs ma) {
    const Q4Args &a = ma.q;
    constexpr int SPG = 4 / NG, PL = WIDE ? 2 : 1;
    __shared__ __align__(16) float red[W * RT * 256];  // [W][RT][16 columns][16 rows]
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int rt0 = blockIdx.x * RT;
    // this workgroup's share of the blocks, and its waves' blocks k0 + wv, k0 + wv + W, ...
    const int ks = blockIdx.y, KS = gridDim.y;
    const int k0 = (int)((int64_t)a.kb_n * ks / KS), k1 = (int)((int64_t)a.kb_n * (ks + 1) / KS);
    const int n_rt = (a.rows + kRow - 1) / kRow;
    const uint8_t *sc_base = a.packed + (size_t)a.n_rec * 1024;
    const uint8_t *zp_base = sc_base + (size_t)a.n_rec * 32 * NG;
    size_t rec0[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int rt = rt0 + t < n_rt ? rt0 + t : n_rt - 1;  // a tile past the end is not stored
        rec0[t] = (size_t)rt * a.kb_n;
    }
    const CodeBits bits;
    f32x4 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};

    uint4 cw[DW][RT];
    Scales<NG> cs[DW][RT];
    uint32_t cz[DW][RT];
    half8 cx[4][PL];
    auto load_w = [&](int st, int kb) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const size_t rec = rec0[t] + kb;
            cw[st][t] = __builtin_bit_cast(
                uint4, __builtin_nontemporal_load(
                           reinterpret_cast<const u32x4_t *>(a.packed + rec * 1024) + lane));
            cs[st][t].load(sc_base + (rec * 16 + 4 * g + (n & 3)) * (2 * NG));
            if (ZP) cz[st][t] = load_zeros<NG>(zp_base + (rec * 16 + n) * NG);
        }
    };
    auto load_x = [&](int w, int kb) {
        const half8 *xp = reinterpret_cast<const half8 *>(ma.xp) + ((size_t)kb * 4 + w) * PL * 64 + lane;
#pragma unroll
        for (int p = 0; p < PL; ++p) cx[w][p] = xp[p * 64];
    };
    if (k0 + wv < k1) {
#pragma unroll
        for (int w = 0; w < 4; ++w) load_x(w, k0 + wv);
    }
#pragma unroll
    for (int d = 0; d < DW; ++d)
        if (k0 + wv + d * W < k1) load_w(d, k0 + wv + d * W);
    auto blocks = [&](auto all, int kb0) {  // as in q4mv_kernel
        constexpr bool ALL = decltype(all)::value;
#pragma unroll
        for (int u = 0; u < DW; ++u) {
            const int kb = kb0 + u * W;
            if (!ALL && kb >= k1) break;
            const int kx = kb + W < k1 ? kb + W : kb;  // the last block's are loaded again
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                f32x4 z[RT];
#pragma unroll
                for (int t = 0; t < RT; ++t) z[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = i * SPG; w < (i + 1) * SPG; ++w) {
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const uint4 q = cw[u][t];
                        const uint32_t word = w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w;
                        const half8 aw = widen(word, bits, Offsets::of<ZP>(cz[u][t] >> (8 * i)));
#pragma unroll
                        for (int p = 0; p < PL; ++p)
                            z[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(aw, cx[w][p], z[t], 0, 0, 0);
                    }
                    load_x(w, kx);  // for the next block, in place
                }
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[t][j] = fmaf(z[t][j], (float)cs[u][t](j, i), acc[t][j]);
            }
            if (ALL || kb + DW * W < k1) load_w(u, kb + DW * W);
        }
    };
    int kb0 = k0 + wv;
    for (; kb0 + (2 * DW - 1) * W < k1; kb0 += DW * W) blocks(std::true_type{}, kb0);
    for (; kb0 < k1; kb0 += DW * W) blocks(std::false_type{}, kb0);
#pragma unroll
    for (int t = 0; t < RT; ++t)
        *reinterpret_cast<f32x4 *>(red + ((wv * RT + t) * 16 + n) * 16 + 4 * g) = acc[t];
    __syncthreads();
    constexpr int ROWS = RT * kRow;
    auto finish = [&](int o, float v) {
        const int b = o / ROWS, row = rt0 * kRow + o % ROWS;
        if (row >= a.rows) return;
        v *= ma.fac[2 * b] * ma.fac[2 * b + 1];
        if (a.bias) v += a.bias[row];
        const size_t at = (size_t)b * a.rows + row;
        if (a.resid) v += a.resid[at];
        a.y[at] = v;
    };
    const int n_out = ROWS * a.B;
    if (KS == 1) {
        for (int o = tid; o < n_out; o += 64 * W)
            finish(o, sum_waves<RT, W, !WIDE>(red, o / ROWS, o % ROWS / 16, o % 16));
        return;
    }
    // The workgroups of these rows leave their sums in the workspace, and the last one to come
    // adds them up, in the order of their columns.  The sums are written and read as agent-scope
    // atomics, which are coherent by themselves: each wave waits for its own stores, the barrier
    // for the waves, and only then is the workgroup counted (no cache write-back is needed).
    float *part = ma.part + (size_t)blockIdx.x * KS * n_out;
    for (int o = tid; o < n_out; o += 64 * W)
        __hip_atomic_store(part + (size_t)ks * n_out + o,
                           sum_waves<RT, W, !WIDE>(red, o / ROWS, o % ROWS / 16, o % 16),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_s_waitcnt(0);
    __shared__ int last;
    __syncthreads();
    if (tid == 0)
        last = __hip_atomic_fetch_add(ma.done + blockIdx.x, 1, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == KS - 1;
    __syncthreads();
    if (!last) return;
    for (int o = tid; o < n_out; o += 64 * W) {
        float v = 0.0f;
        for (int k = 0; k < KS; ++k)
            v += __hip_atomic_load(part + (size_t)k * n_out + o, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        finish(o, v);
    }
}

template <int NG, bool ZP, int B, int RT, int W, int DW>
hipError_t launch_q4mv_one(const Q4Args &a, hipStream_t s) {
    const int n_rt = (a.rows + kRow - 1) / kRow;
    q4mv_kernel<NG, ZP, B, RT, W, DW><<<(n_rt + RT - 1) / RT, 64 * W, 0, s>>>(a);
    return hipGetLastError();
}

// Rows of a workgroup of the product, and how often its columns are cut.  The
// cuts make the number of workgroups fit the 256 compute units: G row groups cut
// KS times take ceil(G KS / 256) rounds of 1 / KS of a row group's work each (one
// workgroup per unit and round; several fit at a time, and the units share the
// memory, so it is a matter of equal shares, not of waves left idle).  Few cuts
// are preferred: each adds a sum to be written and read.  9216 x 8192, five
// tokens: 20.5 us uncut, 18.6 cut in 3 or 4, 19.7 in 8, 23.9 in 16.
// (four tiles a wave share one activation operand at B > 8, where that is 8 KiB a
// block: 36864 x 12288 and sixteen tokens 71 us, with two tiles 83; at B <= 8 the
// smaller shares of two tiles win, 18.6 against 19.5 us)
constexpr int kMmWaves = 4;
constexpr int mm_rt(int B) { return B > 8 ? 4 : 2; }

struct MmShape {
    int groups, cuts;
};

MmShape mm_shape(int rows, int cols, int B) {
    const int kb_n = (cols + kBlk - 1) / kBlk;
    const int per = kRow * mm_rt(B), g = (rows + per - 1) / per;
    const int most = kb_n / kMmWaves < 1 ? 1 : kb_n / kMmWaves > 16 ? 16 : kb_n / kMmWaves;
    int best = 1;
    double cost = 0;
    for (int ks = 1; ks <= most; ++ks) {
        const int64_t wgs = (int64_t)g * ks;
        const double c = (double)((wgs + 255) / 256) / ks + 0.04 * g / 256 * (ks - 1);
        if (ks == 1 || c < cost) {
            best = ks;
            cost = c;
        }
    }
    return {g, best};
}

// Workspace of B > 2: the split activations, two factors a token, the counters
// and, where the columns are cut, the sums.
struct MmWs {
    size_t fac, done, part, total;
};

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

MmWs mm_ws(int rows, int cols, int B) {
    const MmShape sh = mm_shape(rows, cols, B);
    MmWs w;
    w.fac = (size_t)((cols + kBlk - 1) / kBlk) * (B > 8 ? 8192 : 4096);
    w.done = w.fac + 256;
    w.part = w.done + up256((size_t)sh.groups * 4);
    w.total = w.part + (sh.cuts > 1 ? (size_t)sh.groups * sh.cuts * B * mm_rt(B) * kRow * 4 : 0);
    return w;
}

template <int NG, bool ZP>
hipError_t launch_q4_shape(const Q4Args &a, void *ws, hipStream_t s) {
    if (a.B == 1) return launch_q4mv_one<NG, ZP, 1, 1, 8, 2>(a, s);
    if (a.B == 2) return launch_q4mv_one<NG, ZP, 2, 1, 8, 2>(a, s);
    const MmShape sh = mm_shape(a.rows, a.cols, a.B);
    const MmWs w = mm_ws(a.rows, a.cols, a.B);
    uint8_t *base = static_cast<uint8_t *>(ws);
    _Float16 *xp = reinterpret_cast<_Float16 *>(base);
    float *fac = reinterpret_cast<float *>(base + w.fac);
    int *done = reinterpret_cast<int *>(base + w.done);
    q4_split_kernel<<<a.B, kSplitThreads, 0, s>>>(
        SplitArgs{a.x, xp, fac, a.cols, a.kb_n, a.B > 8, a.eps, done, sh.cuts > 1 ? sh.groups : 0});
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const MmArgs m{a, xp, fac, reinterpret_cast<float *>(base + w.part), done};
    const dim3 grid(sh.groups, sh.cuts);
    if (a.B <= 8)
        q4mm_kernel<NG, ZP, false, mm_rt(8), kMmWaves, 1><<<grid, 64 * kMmWaves, 0, s>>>(m);
    else
        q4mm_kernel<NG, ZP, true, mm_rt(16), kMmWaves, 1><<<grid, 64 * kMmWaves, 0, s>>>(m);
    return hipGetLastError();
}

int64_t q4_records(int rows, int cols) {
    return (int64_t)((rows + kRow - 1) / kRow) * ((cols + kBlk - 1) / kBlk);
}

}  // namespace

size_t q4_packed_bytes(int rows, int cols, int group, bool zeros) {
    return (size_t)q4_records(rows, cols) * (1024 + (kBlk / group) * (zeros ? 48 : 32));
}

hipError_t launch_q4_pack(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros,
                          int rows, int cols, int group, uint8_t *packed, hipStream_t s) {
    const int64_t n_rec = q4_records(rows, cols);
    q4_pack_kernel<<<(unsigned)((n_rec + 3) / 4), 256, 0, s>>>(
        codes, scales, zeros, rows, cols, group, (cols + kBlk - 1) / kBlk, n_rec, packed);
    return hipGetLastError();
}

size_t q4_ws_bytes(int rows, int cols, int B) { return B <= 2 ? 0 : mm_ws(rows, cols, B).total; }

hipError_t launch_q4_matvec(const uint8_t *packed, int rows, int cols, int group, bool zeros,
                            const float *x, int B, float eps, const float *bias,
                            const float *resid, float *y, void *ws, hipStream_t s) {
    const Q4Args a{packed, x, bias, resid, y, rows, cols, (cols + kBlk - 1) / kBlk, B,
                   q4_records(rows, cols), eps};
    switch (group) {
        case 32: return zeros ? launch_q4_shape<4, true>(a, ws, s) : launch_q4_shape<4, false>(a, ws, s);
        case 64: return zeros ? launch_q4_shape<2, true>(a, ws, s) : launch_q4_shape<2, false>(a, ws, s);
        default: return zeros ? launch_q4_shape<1, true>(a, ws, s) : launch_q4_shape<1, false>(a, ws, s);
    }
}

}  // namespace spffn
