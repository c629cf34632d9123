// Attention of a tree of drafted tokens over the paged 8-bit cache, many query
// rows: the kernels of fa_cache_prefill.cu with the tree's mask.
#define FA_CACHE_TREE 1
#include "fa_cache_prefill.cu"
