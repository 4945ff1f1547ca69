// kvq_decode_lists.cu -- the split-K decode of kvq_decode_mma.cu over block
// lists (kvq_sparse_decode_attn): the same kernels, compiled with the list
// work items, so the dense ones carry nothing of them.
#define KVQ_DECODE_LISTS 1
#include "kvq_decode_mma.cu"
