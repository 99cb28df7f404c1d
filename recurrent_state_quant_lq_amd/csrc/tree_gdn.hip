// tree_gdn.hip -- drafted token trees of the gated delta rule with a decay per head (gfx950); the kernels are in tree.h.
#define LQ_TREE_KERNELS
#include "tree.h"

namespace lq {
template hipError_t launch_tree_rule<TREE_GDN>(const lq_dims&, const TreeArgs&, hipStream_t);
}  // namespace lq
