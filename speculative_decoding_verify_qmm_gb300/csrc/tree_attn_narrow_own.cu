// The kernel of narrow rows for the own tokens of calls over shared prefixes.
#include "tree_attn_narrow.cuh"

namespace sv {

cudaError_t launch_tree_attn_narrow(const TreeAttnOwnParams& p, cudaStream_t s) { return launch_narrow_any(p, s); }

}  // namespace sv
