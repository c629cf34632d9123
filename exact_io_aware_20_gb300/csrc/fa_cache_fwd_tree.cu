// Attention of a tree of drafted tokens over the paged 8-bit cache, few query
// rows (fa_fwd_cache_tree): the kernels of fa_cache_fwd.cu with the tree's mask.
#define FA_CACHE_TREE 1
#include "fa_cache_fwd.cu"
