// tree_la.hip -- drafted token trees of plain linear attention (gfx950); the kernels are in tree.h.
#define LQ_TREE_KERNELS
#include "tree.h"

namespace lq {
template hipError_t launch_tree_rule<TREE_LA>(const lq_dims&, const TreeArgs&, hipStream_t);
}  // namespace lq
