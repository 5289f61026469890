// Attention over fp16 cache pages: the instances of attn_tile.h.
#include "attn_tile.h"

namespace spffn {

hipError_t launch_attend_f16(const attn::Args &a, bool q16, int dim, int mode, hipStream_t s) {
    return q16 ? attn::launch_all<false, true>(a, dim, mode, s)
               : attn::launch_all<false, false>(a, dim, mode, s);
}

}  // namespace spffn
