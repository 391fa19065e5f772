// kv4_attn.hip -- attention over the paged 4-bit cache, masks by position (gfx950);
// the kernels are in kv4_attn.h.
#include "kv4_attn.h"

namespace rad {

bool kv4_attn_fits(const Kv4Cache &c, const KvBatch &b, int q_heads) {
    return static_cast<int64_t>(attn_shape(b, c, q_heads).plan.pieces) * 64 * kWaves < int64_t(1) << 32;
}

int64_t kv4_attn_workspace(const Kv4Cache &c, const KvBatch &b, int q_heads, int) {
    const Shape s = attn_shape(b, c, q_heads);
    return s.sums + s.stats;
}

hipError_t launch_kv4_attn(const Kv4Cache &c, const KvBatch &b, const Kv4Attn &a, void *workspace, int dtype, hipStream_t st) {
    return launch_attn<false>(c, b, a, workspace, dtype, st);
}

}  // namespace rad
