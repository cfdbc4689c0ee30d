// The kernel of narrow rows for plain calls; those over shared prefixes have theirs in a unit of their own (half a minute to compile each).
#include "tree_attn_narrow.cuh"

namespace sv {

cudaError_t launch_tree_attn_narrow(const TreeAttnParams& p, cudaStream_t s) { return launch_narrow_any(p, s); }

}  // namespace sv
