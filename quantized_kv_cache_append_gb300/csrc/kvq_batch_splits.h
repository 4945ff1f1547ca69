// kvq_batch_splits.h -- the split length of a batch's scored decode, chosen on
// the device from the lengths it finds.
//
// The host knows an upper bound of the lengths; a split length taken from it
// leaves a ragged batch with some odd number of waves of CTAs, the last of
// them nearly empty.  On the device the shortest length is taken whose splits
// are at most as many as the CTAs that were launched, whole waves of them: 16
// sequences of 1024 to 16384 cells (8 heads, int8) take 29 tiles a CTA in one
// wave instead of up to three times 14.  Plain C++ (no CUDA headers), so the
// choice is testable on a host without a GPU.
#pragma once

#ifdef __CUDACC__
#define KVQ_HD __host__ __device__
#else
#define KVQ_HD
#endif

namespace kvq {

constexpr int kBatchMaxSeq = 128;   // sequences a warp holds the lengths of, 4 a lane

// total: tiles of all sequences; items: splits there may be, more than n_seq;
// count(S): splits of S tiles there are, the sum of ceil(tiles / S), at most
// total / S + n_seq.  Returns an S with count(S) <= items, the least or near it.
template <class Count>
KVQ_HD inline int batch_split(long long total, int items, int n_seq, Count count) {
  long long s = (total + items - 1) / items;
  if (s < 1) s = 1;
  for (int i = 0; i < 32; ++i) {
    if (count((int)s) <= items) return (int)s;
    s += 1 + s / 64;
  }
  const long long sure = (total + (items - n_seq) - 1) / (items - n_seq);
  return (int)(s > sure ? s : sure);
}

// Splits per (KV head, row tile) to launch for: the fewest whole waves, up to 4,
// that give a sequence 4 splits in the mean (shorter lengths even out what is
// ragged), else 4; 0: more sequences than that, the host's plan stays.
inline int batch_items(long long capacity, int per, int n_seq) {
  if (n_seq < 2 || n_seq > kBatchMaxSeq) return 0;
  for (int waves = 1; waves <= 4; ++waves) {
    const long long items = waves * capacity / per;
    if (items >= 4LL * n_seq || (waves == 4 && items > n_seq)) return (int)items;
  }
  return 0;
}

}  // namespace kvq
