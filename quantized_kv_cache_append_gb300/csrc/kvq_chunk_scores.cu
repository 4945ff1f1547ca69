// kvq_chunk_scores.cu -- the prompt-chunk attention of kvq_chunk.cu with
// capped, biased and masked scores (kvq_chunk_attn_scored): the same kernel,
// compiled with them, so the plain one carries nothing of them.
#define KVQ_CHUNK_SCORES 1
#include "kvq_chunk.cu"
