// Attention over fp8 (E4M3) cache pages: the instances of attn_tile.h.
#include "attn_tile.h"

namespace spffn {

hipError_t launch_attend_fp8(const attn::Args &a, bool q16, int dim, int mode, hipStream_t s) {
    return q16 ? attn::launch_all<true, true>(a, dim, mode, s)
               : attn::launch_all<true, false>(a, dim, mode, s);
}

}  // namespace spffn
