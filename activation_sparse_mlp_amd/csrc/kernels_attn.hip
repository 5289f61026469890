// Attention over the paged cache: the choice of a launch's shape.
#include "attn_tile.h"

namespace spffn {

hipError_t launch_attend_f16(const attn::Args &a, bool q16, int dim, int mode, hipStream_t s);
hipError_t launch_attend_fp8(const attn::Args &a, bool q16, int dim, int mode, hipStream_t s);

namespace {

struct Shape {
    int mode, wq, cols;  // columns a workgroup takes at a time
};

// max_new tokens of G heads each are the columns a kv head can have.  Few
// columns leave the waves to the tokens (all four take different steps of the
// same columns); many columns take them, up to 128, so that a key is read once.
// At 256 dimensions the outputs of 32 columns would not fit a wave's
// registers: 16 each there.
Shape attn_shape(int G, int dim, int max_new, bool q16) {
    const int cols = max_new * G;
    if (cols <= 8 && !q16) return {attn::kHalf, 1, 8};
    if (cols <= 16) return {attn::kOne, 1, 16};
    if (dim > 128) return cols <= 32 ? Shape{attn::kOne, 2, 32} : Shape{attn::kOne, 4, 64};
    const int wq = cols <= 32 ? 1 : cols <= 64 ? 2 : 4;
    return {attn::kTwo, wq, 32 * wq};
}

}  // namespace

size_t attn_ws_bytes(int heads, int kv_heads, int dim, int max_new, bool q16) {
    const Shape sh = attn_shape(heads / kv_heads, dim, max_new, q16);
    return (size_t)2 * attn::kMaxWgs * sh.cols * (dim + 2) * 4 + attn::kMaxWgs * (sizeof(attn::Task) + sizeof(int));
}

hipError_t launch_tree_attention(const KvCache &c, const AttnCall &q, void *ws, hipStream_t s) {
    const int G = q.heads / c.H;
    const Shape sh = attn_shape(G, c.D, q.max_new, q.q16);
    attn::Args a{};
    a.q = q.q;
    a.out = q.out;
    a.k = c.k;
    a.v = c.v;
    a.ks = c.ks;
    a.vs = c.vs;
    a.starts = q.starts;
    a.lens = q.lens;
    a.table = q.table;
    a.mask = q.mask;
    a.part_o = static_cast<float *>(ws);
    a.part_ml = a.part_o + (size_t)2 * attn::kMaxWgs * sh.cols * c.D;
    a.tasks = reinterpret_cast<attn::Task *>(a.part_ml + (size_t)4 * attn::kMaxWgs * sh.cols);
    a.more = reinterpret_cast<int *>(a.tasks + attn::kMaxWgs);
    a.ldq = q.ldq;
    a.ldo = q.ldo;
    a.scale = q.scale;
    a.N = q.N;
    a.R = q.R;
    a.G = G;
    a.H = c.H;
    a.width = q.width;
    a.pages = c.pages;
    a.shift = c.shift;
    a.max_new = q.max_new;
    // at most this many positions: every table row full, every request max_new tokens
    const int64_t steps = (((int64_t)q.width << c.shift) + 31) / 32 + attn::kSetup;
    const int64_t groups = ((int64_t)q.max_new * G + sh.cols - 1) / sh.cols;
    a.narrow = q.R <= 64 && steps * groups * c.H * q.R < (int64_t)1 << 31;
    a.wq = sh.wq;
    a.clear = q.clear;
    return c.fp8 ? launch_attend_fp8(a, q.q16, c.D, sh.mode, s)
                 : launch_attend_f16(a, q.q16, c.D, sh.mode, s);
}

}  // namespace spffn
