// kvq_decode_scores.cu -- the split-K decode of kvq_decode_mma.cu with capped,
// biased and windowed scores (kvq_decode_attn_scored): the same kernels,
// compiled with them, so the dense ones carry nothing of them.
#define KVQ_DECODE_SCORES 1
#include "kvq_decode_mma.cu"
