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
// Append.  Each workgroup takes 16 tokens of one head, keys or values.
//   keys:   a thread converts one packet (E head dimensions of a token) and
//           stores it with one 16-byte store, tokens fastest, so that tokens of
//           neighbouring slots write neighbouring packets;
//   values: a packet is E neighbouring slots of one dimension.  Tokens whose
//           slots run on inside a packet are written together: the first of
//           the run (its packet's first slot, or one whose predecessor in the
//           input is not the slot before) takes all of it, each lane one
//           dimension, a whole packet as one 16-byte store and a part of one
//           element by element.  A decode step's tokens are runs of one.
// HBM bounds long inputs (each element is read once and written once), the
// launch short ones.  The conversion is one rounding: fp16 to nearest, fp8 the
// nearest E4M3 value of x / scale (an fp32 division), saturating at +-448 (NaN
// stays NaN).
// ---------------------------------------------------------------------------
constexpr int kAppTokens = 16;

struct AppArgs {
    const void *k, *v;
    uint8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *slots;
    int64_t ldk, ldv;
    int N, H, D, shift;
    int64_t n_slots;
};

__device__ __forceinline__ float e4m3_clamp(float v) {
    return v > 448.0f ? 448.0f : v < -448.0f ? -448.0f : v;  // NaN passes
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(a), e4m3_clamp(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(c), e4m3_clamp(d), w, true);
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

template <bool FP8, bool SRC16>
__global__ __launch_bounds__(256) void kv_append_kernel(AppArgs a) {
    constexpr int E = FP8 ? 16 : 8;
    typedef typename std::conditional<SRC16, _Float16, float>::type S;
    const int n0 = blockIdx.x * kAppTokens, h = blockIdx.y;
    const int ps = 1 << a.shift;
    if (blockIdx.z == 0) {
        const float ks = FP8 ? a.ks[h] : 1.0f;
        const int npk = a.D / E;
        for (int i = threadIdx.x; i < npk * kAppTokens; i += 256) {
            const int n = n0 + (i & (kAppTokens - 1)), pk = i / kAppTokens;
            if (n >= a.N) continue;
            const int slot = a.slots[n];
            if (slot < 0 || slot >= a.n_slots) continue;
            const S *src = static_cast<const S *>(a.k) + (size_t)n * a.ldk + (size_t)h * a.D + pk * E;
            float v[E];
            if constexpr (SRC16) {
#pragma unroll
                for (int q = 0; q < E / 8; ++q) {
                    const half8 x = reinterpret_cast<const half8 *>(src)[q];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[8 * q + e] = (float)x[e];
                }
            } else {
#pragma unroll
                for (int q = 0; q < E / 4; ++q) {
                    const float4 x = reinterpret_cast<const float4 *>(src)[q];
                    v[4 * q] = x.x;
                    v[4 * q + 1] = x.y;
                    v[4 * q + 2] = x.z;
                    v[4 * q + 3] = x.w;
                }
            }
            if (FP8) {
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = v[e] / ks;
            }
            const size_t page = (size_t)(slot >> a.shift), o = (size_t)(slot & (ps - 1));
            const size_t at = ((page * a.H + h) * npk + pk) * ps + o;
            reinterpret_cast<uint4 *>(a.kc)[at] = to_packet<FP8>(v);
        }
        return;
    }
    const float vs = FP8 ? a.vs[h] : 1.0f;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    for (int t = 0; t < kAppTokens / 4; ++t) {
        const int n = n0 + wv * (kAppTokens / 4) + t;
        if (n >= a.N) break;
        const int slot = a.slots[n];
        if (slot < 0 || slot >= a.n_slots) continue;
        const int o = slot & (E - 1);
        if (o != 0 && n > 0 && a.slots[n - 1] == slot - 1) continue;  // inside a run
        bool runs = false;
        if (lane < E - o && n + lane < a.N) runs = a.slots[n + lane] == slot + lane;
        const int m = __ffsll((long long)~__ballot(runs)) - 1;  // >= 1: lane 0 is the slot itself
        const size_t page = (size_t)(slot >> a.shift);
        const size_t row = (page * a.H + h) * (size_t)(ps / E) + ((slot & (ps - 1)) / E);
        for (int d = lane; d < a.D; d += 64) {
            const S *src = static_cast<const S *>(a.v) + (size_t)n * a.ldv + (size_t)h * a.D + d;
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[e] = e < m ? (float)src[(size_t)e * a.ldv] : 0.0f;
                if (FP8) v[e] = v[e] / vs;
            }
            const uint4 pkt = to_packet<FP8>(v);
            uint8_t *dst = a.vc + (row * a.D + d) * 16;
            if (m == E) {
                *reinterpret_cast<uint4 *>(dst) = pkt;
            } else {
                const uint32_t w[4] = {pkt.x, pkt.y, pkt.z, pkt.w};
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (e >= m) continue;
                    if constexpr (FP8) dst[o + e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
                    else reinterpret_cast<uint16_t *>(dst)[o + e] =
                            (uint16_t)(w[e / 2] >> (16 * (e % 2)));
                }
            }
        }
    }
}

hipError_t launch_kv_append(const KvCache &c, const void *k, const void *v, bool src16, int64_t ldk,
                            int64_t ldv, const int32_t *slots, int N, hipStream_t s) {
    AppArgs a{k, v, c.k, c.v, c.ks, c.vs, slots, ldk, ldv, N, c.H, c.D, c.shift,
              (int64_t)c.pages << c.shift};
    const dim3 grid((N + kAppTokens - 1) / kAppTokens, c.H, 2);
    if (c.fp8) {
        if (src16) kv_append_kernel<true, true><<<grid, 256, 0, s>>>(a);
        else kv_append_kernel<true, false><<<grid, 256, 0, s>>>(a);
    } else {
        if (src16) kv_append_kernel<false, true><<<grid, 256, 0, s>>>(a);
        else kv_append_kernel<false, false><<<grid, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace spffn
