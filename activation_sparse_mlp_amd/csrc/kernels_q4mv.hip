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
//     a nibble under the exponent of 1024 reads as 1024 + q (or 1024 + 16 q),
//     and one packed operation takes 1024 + z off (or divides by 16 and takes
//     64 + z off), so eight codes cost nine instructions.  The scale is applied
//     in fp32 to the product of its group, so no weight is ever rounded;
//   * activations are the B operand, hi + lo halves of x scaled by a power of
//     two per token and block of 128 columns (largest magnitude in [2^14,
//     2^15)): about 22 significant bits down to 2^-18 of the block's largest,
//     an absolute 2^-40 of it below.  For B <= 8 the hi halves are columns 0..7
//     and the lo halves columns 8..15 of one instruction, for B > 8 they take one
//     each into the same accumulator;
//   * a wave owns whole blocks of 128 columns (wave, wave + W, ...) of RT tiles
//     of 16 rows, so it splits each activation once and no wave waits for
//     another before the final sum over the workgroup's waves, which is taken
//     in a fixed order.  The RMS scale needs no pass of its own: it has no gain,
//     so it is one factor per token at the end, and each wave already holds the
//     activations whose squares it sums.
//
// Packed layout (launch_q4_pack): per tile of 16 rows and block of 128 columns
// 1 KiB of codes in the order of one wave's 16-byte loads -- lane l = 16 g + m
// holds row m, word w the eight columns 32 w + 8 g + e, code 2i in nibble i and
// code 2i + 1 in nibble i + 4 -- then all scales [tile, block, group, 16] fp16,
// then all zero points (same shape, bytes).  Rows and columns are padded with
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
        const size_t at = ((size_t)rec * ng + gi) * 16 + m;
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

// Eight codes as q - z.  off = -(1024 + z), off16 = -(64 + z), both twice.
__device__ __forceinline__ half8 widen(uint32_t w, half2v off, half2v off16) {
    const half2v sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t k1 = 0x64006400u;
    const uint32_t h = w >> 8;
    const half2v a = __builtin_bit_cast(half2v, (w & 0x000F000Fu) | k1) + off;
    const half2v b = __builtin_elementwise_fma(__builtin_bit_cast(half2v, (w & 0x00F000F0u) | k1),
                                               sixteenth, off16);
    const half2v c = __builtin_bit_cast(half2v, (h & 0x000F000Fu) | k1) + off;
    const half2v d = __builtin_elementwise_fma(__builtin_bit_cast(half2v, (h & 0x00F000F0u) | k1),
                                               sixteenth, off16);
    half8 r;
    r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
    r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
    return r;
}

template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF,
                                                               false)));
}

// The largest value of each group of LPT (16, 32 or 64) lanes, in every lane of it.
template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
    v = dpp_max<0xB1>(v);
    v = dpp_max<0x4E>(v);
    v = dpp_max<0x141>(v);
    v = dpp_max<0x140>(v);
    if constexpr (LPT >= 32) v = fmaxf(v, __shfl_xor(v, 16, 64));
    if constexpr (LPT >= 64) v = fmaxf(v, __shfl_xor(v, 32, 64));
    return v;
}

// NG: groups per block (128 / group size).  WIDE: B > 8.  E: activations per
// lane and pass (2: B = 1, 4: B = 2, 8: more), so a pass takes E / 2 tokens.
template <int NG, bool ZP, bool WIDE, int E, int RT, int W>
__global__ __launch_bounds__(64 * W) void q4mv_kernel(Q4Args a) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int LPT = kBlk / E;             // lanes per token
    constexpr int TP = 64 / LPT;              // tokens per pass
    constexpr int NP = WIDE ? 4 : E == 8 ? 2 : 1;
    constexpr int SPG = 4 / NG;               // instructions per group
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int n = lane & 15, g = lane >> 4;
    const int rt0 = blockIdx.x * RT;
    const int n_rt = (a.rows + kRow - 1) / kRow;
    const int B = a.B;

    // this wave's staging area: hi and lo planes of B tokens, then 16 factors
    _Float16 *xh = reinterpret_cast<_Float16 *>(smem) + (size_t)wv * (2 * B * kXPitch + 32);
    _Float16 *xl = xh + B * kXPitch;
    float *xf = reinterpret_cast<float *>(xl + B * kXPitch);

    const uint8_t *sc_base = a.packed + (size_t)a.n_rec * 1024;
    const uint8_t *zp_base = sc_base + (size_t)a.n_rec * 32 * NG;

    size_t rec0[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int rt = rt0 + t < n_rt ? rt0 + t : n_rt - 1;  // a tile past the end is not stored
        rec0[t] = (size_t)rt * a.kb_n;
    }

    const int tl = lane / LPT, el = (lane % LPT) * E;  // token of a pass, first column
    const int col_tok = WIDE ? (n < B ? n : B - 1) : ((n & 7) < B ? (n & 7) : B - 1);
    const _Float16 *bsrc = (!WIDE && n >= 8 ? xl : xh) + col_tok * kXPitch + 8 * g;
    const _Float16 *bsrc_lo = xl + col_tok * kXPitch + 8 * g;

    f32x4 acc[RT];
    float ss[NP];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < NP; ++p) ss[p] = 0.0f;

    uint4 cw[RT];
    half4 cs[RT][NG];
    uint32_t cz[RT][NG];
    float cx[NP][E];
    auto load = [&](int kb) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const size_t rec = rec0[t] + kb;
            cw[t] = __builtin_bit_cast(
                uint4, __builtin_nontemporal_load(
                           reinterpret_cast<const u32x4_t *>(a.packed + rec * 1024) + lane));
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                cs[t][i] = *reinterpret_cast<const half4 *>(sc_base + (rec * NG + i) * 32 + g * 8);
                if (ZP) cz[t][i] = zp_base[(rec * NG + i) * 16 + n];
            }
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int tok = p * TP + tl, c = kb * kBlk + el;
            const bool in = tok < B && c < a.cols;  // cols % 32 == 0: all E columns or none
            const float *src = a.x + (size_t)(in ? tok : 0) * a.cols + (in ? c : 0);
            if constexpr (E == 2) {
                const float2 v = *reinterpret_cast<const float2 *>(src);
                cx[p][0] = in ? v.x : 0.0f;
                cx[p][1] = in ? v.y : 0.0f;
            } else {
#pragma unroll
                for (int q = 0; q < E / 4; ++q) {
                    const float4 v = reinterpret_cast<const float4 *>(src)[q];
                    cx[p][4 * q + 0] = in ? v.x : 0.0f;
                    cx[p][4 * q + 1] = in ? v.y : 0.0f;
                    cx[p][4 * q + 2] = in ? v.z : 0.0f;
                    cx[p][4 * q + 3] = in ? v.w : 0.0f;
                }
            }
        }
    };

    if (wv < a.kb_n) load(wv);
    for (int kb = wv; kb < a.kb_n; kb += W) {
        uint4 w4[RT];
        half4 s4[RT][NG];
        uint32_t z4[RT][NG];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            w4[t] = cw[t];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                s4[t][i] = cs[t][i];
                if (ZP) z4[t][i] = cz[t][i];
            }
        }
        // ---- split this block's activations into the wave's LDS planes ----
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int tok = p * TP + tl;
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                m = fmaxf(m, fabsf(cx[p][e]));
                ss[p] = fmaf(cx[p][e], cx[p][e], ss[p]);
            }
            m = lanes_max<LPT>(m);
            const bool inf = __float_as_uint(m) >= 0x7F800000u;
            if (__any(inf)) {
                // an infinity: scale by the finite values, and keep it out of lo
                float f = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float v = fabsf(cx[p][e]);
                    f = fmaxf(f, v < __builtin_inff() ? v : 0.0f);
                }
                f = lanes_max<LPT>(f);
                if (inf) m = f;
            }
            uint32_t eb = __float_as_uint(m) >> 23;
            eb = eb < 16 ? 16 : eb;
            const float up = __uint_as_float((268u - eb) << 23);
            if (tok < B) {
                _Float16 hi[E], lo[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float v = cx[p][e] * up;
                    hi[e] = (_Float16)v;
                    const float rest = v - (float)hi[e];
                    lo[e] = (_Float16)(fabsf(v) < __builtin_inff() ? rest : 0.0f);
                }
                _Float16 *dh = xh + tok * kXPitch + el, *dl = xl + tok * kXPitch + el;
                if constexpr (E == 2) {
                    *reinterpret_cast<half2v *>(dh) = half2v{hi[0], hi[1]};
                    *reinterpret_cast<half2v *>(dl) = half2v{lo[0], lo[1]};
                } else if constexpr (E == 4) {
                    *reinterpret_cast<half4 *>(dh) = half4{hi[0], hi[1], hi[2], hi[3]};
                    *reinterpret_cast<half4 *>(dl) = half4{lo[0], lo[1], lo[2], lo[3]};
                } else {
                    *reinterpret_cast<half8 *>(dh) =
                        half8{hi[0], hi[1], hi[2], hi[3], hi[4], hi[5], hi[6], hi[7]};
                    *reinterpret_cast<half8 *>(dl) =
                        half8{lo[0], lo[1], lo[2], lo[3], lo[4], lo[5], lo[6], lo[7]};
                }
                if (el == 0) xf[tok] = __uint_as_float((eb - 14u) << 23);
            }
        }
        if (kb + W < a.kb_n) load(kb + W);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        half8 bh[4], bl[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            bh[w] = *reinterpret_cast<const half8 *>(bsrc + 32 * w);
            if (WIDE) bl[w] = *reinterpret_cast<const half8 *>(bsrc_lo + 32 * w);
        }
        const float f = xf[col_tok];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const uint32_t words[4] = {w4[t].x, w4[t].y, w4[t].z, w4[t].w};
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                half2v off = {(_Float16)-1032.0f, (_Float16)-1032.0f};
                half2v off16 = {(_Float16)-72.0f, (_Float16)-72.0f};
                if (ZP) {
                    const _Float16 zp = (_Float16)(float)z4[t][i];
                    off = half2v{(_Float16)-1024.0f - zp, (_Float16)-1024.0f - zp};
                    off16 = half2v{(_Float16)-64.0f - zp, (_Float16)-64.0f - zp};
                }
                f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = i * SPG; w < (i + 1) * SPG; ++w) {
                    const half8 aw = widen(words[w], off, off16);
                    z = __builtin_amdgcn_mfma_f32_16x16x32_f16(aw, bh[w], z, 0, 0, 0);
                    if (WIDE) z = __builtin_amdgcn_mfma_f32_16x16x32_f16(aw, bl[w], z, 0, 0, 0);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[t][j] = fmaf(z[j], (float)s4[t][i][j] * f, acc[t][j]);
                }
            }
        }
        __builtin_amdgcn_wave_barrier();  // the next block's split overwrites these planes
    }

    // ---- fixed-order sum over the workgroup's waves, scale, bias, residual ----
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);            // [W][RT][16 columns][16 rows]
    float *sq = red + W * RT * 256;                          // [W][16] sums of squares
#pragma unroll
    for (int t = 0; t < RT; ++t)
        *reinterpret_cast<f32x4 *>(red + ((wv * RT + t) * 16 + n) * 16 + 4 * g) = acc[t];
    if (a.eps >= 0.0f) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            float v = ss[p];
            for (int o = 1; o < LPT; o <<= 1) v += __shfl_xor(v, o, 64);
            const int tok = p * TP + tl;
            if (el == 0 && tok < B) sq[wv * 16 + tok] = v;
        }
    }
    __syncthreads();
    for (int o = tid; o < RT * kRow * B; o += 64 * W) {
        const int b = o / (RT * kRow), lr = o - b * (RT * kRow), t = lr >> 4, r = lr & 15;
        const int row = rt0 * kRow + lr;
        if (row >= a.rows) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            v += red[((w * RT + t) * 16 + b) * 16 + r];
            if (!WIDE) v += red[((w * RT + t) * 16 + b + 8) * 16 + r];
        }
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

template <int NG, bool ZP, bool WIDE, int E, int RT, int W>
hipError_t launch_q4mv_one(const Q4Args &a, hipStream_t s) {
    const int n_rt = (a.rows + kRow - 1) / kRow;
    const size_t stage = (size_t)W * (2 * a.B * kXPitch + 32) * 2;
    const size_t red = (size_t)W * RT * 1024 + (size_t)W * 64;
    const size_t lds = stage > red ? stage : red;
    auto fn = q4mv_kernel<NG, ZP, WIDE, E, RT, W>;
    if (lds > 65536) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    fn<<<(n_rt + RT - 1) / RT, 64 * W, lds, s>>>(a);
    return hipGetLastError();
}

template <int NG, bool ZP, int RT, int W>
hipError_t launch_q4mv_b(const Q4Args &a, hipStream_t s) {
    if (a.B > 8) return launch_q4mv_one<NG, ZP, true, 8, RT, W>(a, s);
    if (a.B > 2) return launch_q4mv_one<NG, ZP, false, 8, RT, W>(a, s);
    if (a.B == 2) return launch_q4mv_one<NG, ZP, false, 4, RT, W>(a, s);
    return launch_q4mv_one<NG, ZP, false, 2, RT, W>(a, s);
}

template <int RT, int W>
hipError_t launch_q4mv_g(const Q4Args &a, int group, bool zp, hipStream_t s) {
    switch (group) {
        case 32: return zp ? launch_q4mv_b<4, true, RT, W>(a, s) : launch_q4mv_b<4, false, RT, W>(a, s);
        case 64: return zp ? launch_q4mv_b<2, true, RT, W>(a, s) : launch_q4mv_b<2, false, RT, W>(a, s);
        default: return zp ? launch_q4mv_b<1, true, RT, W>(a, s) : launch_q4mv_b<1, false, RT, W>(a, s);
    }
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

hipError_t launch_q4_matvec(const uint8_t *packed, int rows, int cols, int group, bool zeros,
                            const float *x, int B, float eps, const float *bias,
                            const float *resid, float *y, hipStream_t s) {
    const int n_rt = (rows + kRow - 1) / kRow;
    Q4Args a{packed, x, bias, resid, y, rows, cols, (cols + kBlk - 1) / kBlk, B,
             q4_records(rows, cols), eps};
    // two tiles per wave halve the work of splitting the activations; one tile
    // per wave where two would leave compute units without a workgroup
    if (n_rt >= 512) return launch_q4mv_g<2, 8>(a, group, zeros, s);
    return launch_q4mv_g<1, 8>(a, group, zeros, s);
}

}  // namespace spffn
