// kv4_attn_tree.hip -- attention for trees of drafted tokens over the paged 4-bit
// cache (gfx950); the kernels are in kv4_attn.h.
#include "kv4_attn.h"

namespace rad {

hipError_t launch_kv4_attn_tree(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, void *workspace, int dtype, hipStream_t st) {
    return launch_attn<true>(c, b, a, workspace, dtype, st);
}

}  // namespace rad
