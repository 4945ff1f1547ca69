// kvq_select.cu -- the blocks each query token and KV head attends to
// (kvq_select_blocks): a score for every block from its key bounds, and the
// n_sel highest.
//
// The score estimates the largest q . k over a block's keys: per dim the larger
// of q lo and q hi, i.e. max(q, 0) hi + min(q, 0) lo, an upper bound for the q
// it is computed with.  That q is rounded to int8 codes with a power-of-two
// scale per 64 dims and the bounds are such codes, so a group's sum S is a
// whole number below 2^21 and S * scale_q * scale_k is exact in fp32; 2 or 4
// groups are added pairwise in fp32, and the query heads of a KV head give
// their maximum.  No sum depends on its order, so the chosen blocks do not
// depend on how the work is split; ties go to the lower block.
//
// One cluster of CTAs per (sequence, KV head, up to 32 query rows); its CTAs
// share the visible blocks, a warp scores 16 at a time:
//
//   scores     mma.sync.m16n8k16, 16 blocks x 8 query rows, the codes as fp16
//              (exact: whole numbers below 128, sums below 2^21 in fp32).
//              The dims of a k-step are free to choose, so a lane's 16-byte
//              loads of 16 consecutive dims are its A fragments of 4
//              k-steps: no shared memory, no shuffles.  lo against min(c, 0)
//              and hi against max(c, 0) add up in one accumulator per 64
//              dims.  (dp4a, which the codes suggest, runs at 8 lanes a
//              cycle and SM on this chip: 64 sequences took 121 us in it.)
//   keys       the score as an order-preserving integer goes straight to the
//              shared memory of the CTA that leads its token's selection
//              (distributed shared memory)
//   selection  after one cluster barrier each leader counts its keys in bins
//              of equal score width, compares those of the bin that holds
//              the n_sel-th largest, and writes the list in ascending order
//
// One GB300: 512 blocks x 8 heads 6.2 us (launch, three dependent loads and 2.5
// us of selection), 4096 blocks x 8 heads x 4 tokens 12.6 us, 64 sequences of
// 129 to 4096 blocks x 8 heads 70 us (4.1 TB/s of bounds, 60 % of the measured
// copy rate; an SM holds 24 warps, which spend a third of their time on the
// dependent loads before a row's first score and on its selection).
//
// A token's query rows are padded to a power of two (or a multiple of 8) by
// repeating its last row, which leaves the maximum as it is.
#include <math.h>
#include <stdint.h>

#include "kvq_internal.cuh"
#include "kvq_ptx.cuh"

namespace kvq {
namespace {

constexpr int kOrderRegs = 4;               // up to 128 sequences are ordered by length,
constexpr int kOrderSteps = 4;              // in so many steps of max_ctx
constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kForced = 0xffffffffu;   // keys: 0 not a candidate, kForced always kept

// The smallest e with 127 * 2^e >= m (m >= 0, finite or inf), in [-60, 60].
__device__ __forceinline__ int q_exponent(float m) {
  const uint32_t b = __float_as_uint(m);
  const int e = (int)(b >> 23) - 126 - 7 + ((b & 0x7fffffu) > 0x7e0000u);
  return min(max(e, -60), 60);
}

__device__ __forceinline__ float pow2f_exact(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// A score -> uint32 in the same order, clear of 0 and kForced; -0 counts as
// +0.  Scores of kvq_bound_blocks's scales stay below 2^100; what other
// scales may give is held to +-1e38 (NaN: the lowest), so differences of
// scores are finite below.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(fminf(fmaxf(x, -1e38f), 1e38f) + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 4 int8 codes of one word -> two fp16 pairs, exactly: 0x6400 | (c ^ 0x80) is
// 1152 + c.
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  lo = hsub2(prmt(w, 0x64646464u, 0x4140u), 0x64806480u);
  hi = hsub2(prmt(w, 0x64646464u, 0x4342u), 0x64806480u);
}

// Layout of the dynamic shared memory: the q codes as B fragments
// [n-tile][64-dim group][k-step 0..3][lo, hi][lane][2 words], the q scales
// [row][group] fp32, the keys [lead row][key_row].
//
// Keys of one token, padded to whole 16-byte reads.
__host__ __device__ inline int key_row(int n_cap) { return (n_cap + 3) / 4 * 4; }
struct SelSmem {
  int scales, keys, bytes;
};
__host__ __device__ inline SelSmem sel_smem(int hd, int nt, int lead_rows, int n_cap) {
  const int ng = hd / kGroup;
  SelSmem m;
  m.scales = nt * ng * 8 * 256;
  m.keys = m.scales + nt * 8 * ng * 4;
  m.bytes = m.keys + lead_rows * key_row(n_cap) * 4;
  return m;
}

// Which of keys[0 .. n) are the k largest: every key above `thr`, and the
// first `ties` of those equal to it (in index order).  Keys of 0 are never
// taken.  All threads call it; the result is the same in all.
struct Threshold {
  uint32_t thr;
  uint32_t ties;
  int count;      // how many are taken
};

// Scratch of a selection: bins and ranked keys while the threshold is sought,
// then the list's entries (16 bits each: indexes stay below 32768).
constexpr int kBins = 512, kBinBits = 9, kBinsPL = kBins / 32;   // (kBinsPL: bins a lane sums)
constexpr int kRanks = 3584;
constexpr int kListMax = 2 * (kBins + kRanks);
struct alignas(16) SelScratch {
  union {
    struct {
      uint32_t hist[kBins];
      uint32_t rank[kRanks];
    };
    uint16_t list[kListMax];
  };
  uint32_t sums[2][3][16];    // what the warps tell one another, two rounds in turn
  uint4 found;                // bin, what is left to take in it, its keys
  uint32_t n_rank;
  int last;                   // the last visible block is in the list
};

// Sums over the CTA, one barrier each.
template <int THREADS>
struct Team {
  static constexpr int warps = THREADS / 32;
  SelScratch& sc;
  int round = 0;

  __device__ __forceinline__ uint32_t sum(uint32_t v) {
    v = __reduce_add_sync(kAll, v);
    uint32_t* s = sc.sums[round][0];
    round ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < warps; w += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(s + w);
      v += (x.x + x.y) + (x.z + x.w);
    }
    return v;
  }
  // the sum, and lo's minimum and hi's maximum
  __device__ __forceinline__ uint32_t sum_range(uint32_t v, uint32_t& lo, uint32_t& hi) {
    lo = __reduce_min_sync(kAll, lo);
    hi = __reduce_max_sync(kAll, hi);
    uint32_t (*s)[16] = sc.sums[round];
    if ((threadIdx.x & 31) == 0) {
      s[1][threadIdx.x >> 5] = lo;
      s[2][threadIdx.x >> 5] = hi;
    }
    v = sum(v);
#pragma unroll
    for (int w = 0; w < warps; w += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(s[1] + w), y = *reinterpret_cast<const uint4*>(s[2] + w);
      lo = min(min(min(lo, x.x), min(x.y, x.z)), x.w);
      hi = max(max(max(hi, y.x), max(y.y, y.z)), y.w);
    }
    return v;
  }
  // exclusive prefix sum over the threads
  __device__ __forceinline__ uint32_t before(uint32_t v) {
    const int lane = threadIdx.x & 31, me = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += y;
    }
    uint32_t* s = sc.sums[round][0];
    round ^= 1;
    if (lane == 31) s[me] = incl;
    __syncthreads();
    uint32_t base = 0;
#pragma unroll
    for (int w = 0; w < warps; w += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(s + w);
      base += (w < me ? x.x : 0u) + (w + 1 < me ? x.y : 0u) + (w + 2 < me ? x.z : 0u) + (w + 3 < me ? x.w : 0u);
    }
    return base + incl - v;
  }
};

// A thread's run of consecutive keys, read from shared memory in every pass.
// Runs are a multiple of 4 long; keys past n read as 0.  (Kept in registers,
// unrolled, the passes took longer: this code runs once per CTA, and its
// length costs more than its loads.)
template <int THREADS>
struct KeyRun {
  const uint32_t* keys;
  int first, len, n;

  __device__ __forceinline__ KeyRun(const uint32_t* k, int count) : keys(k), n(count) {
    len = (count + 4 * THREADS - 1) / (4 * THREADS) * 4;
    first = threadIdx.x * len;
  }
  // f(quad, index of its first key)
  template <class F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll 1
    for (int i = first; i < min(first + len, n); i += 4) {
      uint4 v = *reinterpret_cast<const uint4*>(keys + i);   // (rows are padded to 4)
      if (i + 1 >= n) v.y = 0;
      if (i + 2 >= n) v.z = 0;
      if (i + 3 >= n) v.w = 0;
      f(v, i);
    }
  }
};

// The k largest keys: bins of equal score width count them (scores are spread
// like a bell, so the k-th falls among a few), the keys of the bin that holds
// the k-th are listed and compared with one another.  A bin still too full
// for that (long ties) is cut again in key units, until one value is left.
template <int THREADS>
__device__ __forceinline__ Threshold find_threshold(Team<THREADS>& team, const KeyRun<THREADS>& run, int k,
                                                    SelScratch& sc) {
  const int tid = threadIdx.x, lane = tid & 31;
  // counts of candidates and forced ones, range of the others
  uint32_t kmin = 0xffffffffu, kmax = 0, both = 0;
  run.each([&](const uint4& v, int) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t x = c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w;
      both += (x != 0 ? 1u : 0u) + (x == kForced ? 0x10000u : 0u);   // (below 2^15 + 1 keys each)
      kmin = min(kmin, x - 1u);               // 0 counts as the highest,
      kmax = max(kmax, x + 1u);               // kForced as the lowest
    }
  });
  uint4* hist4 = reinterpret_cast<uint4*>(sc.hist);
  auto clear = [&]() {
#pragma unroll
    for (int j = tid; j < kBins / 4; j += THREADS) hist4[j] = make_uint4(0, 0, 0, 0);
    if (tid == 0) sc.n_rank = 0;
  };
  clear();
  both = team.sum_range(both, kmin, kmax);
  ++kmin;
  --kmax;
  const int cand = (int)(both & 0xffffu), forced = (int)(both >> 16);
  if (cand <= k) return {0u, 0u, cand};                     // all of them
  if (forced >= k) return {kForced, (uint32_t)k, k};
  uint32_t rem = (uint32_t)(k - forced);                    // 1 <= rem < keys in [kmin, kmax]
  bool linear = true;
  for (;;) {
    if (kmin == kmax) return {kmin, rem, k};
    // bin = the whole number nearest (score - lowest) * width + 1, read off
    // the mantissa of a sum with 2^23; it never falls with the score
    const float f0 = score_of(kmin);
    const float width = __fdividef((float)(kBins - 4), score_of(kmax) - f0);
    const int shift = max(0, 32 - __clz(kmax - kmin) - kBinBits);
    auto bin_of = [&](uint32_t x) -> uint32_t {   // kBins: outside the range
      const uint32_t lin = min(__float_as_uint(fmaf(score_of(x) - f0, width, 8388609.0f)) - 0x4b000000u, (uint32_t)kBins - 1);
      return x - kmin <= kmax - kmin ? (linear ? lin : (x - kmin) >> shift) : (uint32_t)kBins;
    };
    run.each([&](const uint4& v, int) {
      const uint32_t b0 = bin_of(v.x), b1 = bin_of(v.y), b2 = bin_of(v.z), b3 = bin_of(v.w);
      if (b0 < kBins) atomicAdd(&sc.hist[b0], 1u);
      if (b1 < kBins) atomicAdd(&sc.hist[b1], 1u);
      if (b2 < kBins) atomicAdd(&sc.hist[b2], 1u);
      if (b3 < kBins) atomicAdd(&sc.hist[b3], 1u);
    });
    __syncthreads();
    if (tid < 32) {
      // lane l sums the bins from kBinsPL (31 - l) up, so lanes run from the
      // top down; then the lane that holds the rem-th largest is scanned the
      // same way, a bin a lane
      uint32_t sum = 0;
#pragma unroll
      for (int j = 0; j < kBinsPL / 4; ++j) {
        const uint4 v = hist4[(31 - lane) * (kBinsPL / 4) + j];
        sum += (v.x + v.y) + (v.z + v.w);
      }
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += y;
      }
      const int src = __ffs(__ballot_sync(kAll, incl >= rem)) - 1;
      const uint32_t left = rem - __shfl_sync(kAll, incl - sum, src);
      const uint32_t c = lane < kBinsPL ? sc.hist[(32 - src) * kBinsPL - 1 - lane] : 0u;
      incl = c;
#pragma unroll
      for (int o = 1; o < kBinsPL; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += y;
      }
      const int at = __ffs(__ballot_sync(kAll, incl >= left)) - 1;
      if (lane == at) sc.found = make_uint4((uint32_t)((32 - src) * kBinsPL - 1 - at), left - (incl - c), c, 0);
    }
    __syncthreads();
    const uint32_t bin = sc.found.x, m = sc.found.z;
    rem = sc.found.y;
    if (m <= (uint32_t)kRanks) {
      // list the bin's keys, then find the one with fewer than rem above it
      // and at least rem at or above it
      run.each([&](const uint4& v, int) {
        const bool h0 = bin_of(v.x) == bin, h1 = bin_of(v.y) == bin;
        const bool h2 = bin_of(v.z) == bin, h3 = bin_of(v.w) == bin;
        if (h0 || h1 || h2 || h3) {   // (rare)
          if (h0) sc.rank[atomicAdd(&sc.n_rank, 1u)] = v.x;
          if (h1) sc.rank[atomicAdd(&sc.n_rank, 1u)] = v.y;
          if (h2) sc.rank[atomicAdd(&sc.n_rank, 1u)] = v.z;
          if (h3) sc.rank[atomicAdd(&sc.n_rank, 1u)] = v.w;
        }
      });
      __syncthreads();
      auto place = [&](uint32_t x, uint32_t& gt, uint32_t& ge) {
        gt = ge = 0;
#pragma unroll 4
        for (uint32_t j = 0; j < m; ++j) {
          const uint32_t y = sc.rank[j];
          gt += y > x;
          ge += y >= x;
        }
      };
      uint32_t gt, ge;
      if (m <= 32) {   // each warp by itself
        const uint32_t x = (uint32_t)lane < m ? sc.rank[lane] : 0u;
        place(x, gt, ge);
        const int s = __ffs(__ballot_sync(kAll, x != 0 && gt < rem && ge >= rem)) - 1;
        return {__shfl_sync(kAll, x, s), rem - __shfl_sync(kAll, gt, s), k};
      }
      for (uint32_t i = (int)threadIdx.x; i < m; i += THREADS) {
        const uint32_t x = sc.rank[i];
        place(x, gt, ge);
        if (gt < rem && ge >= rem) {   // (equal keys write the same)
          sc.found.x = x;
          sc.found.y = rem - gt;
        }
      }
      __syncthreads();
      return {sc.found.x, sc.found.y, k};
    }
    // the range of the bin's keys, for the next round
    uint32_t lo = 0xffffffffu, hi = 0;
    run.each([&](const uint4& v, int) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t x = c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w;
        if (bin_of(x) == bin) {
          lo = min(lo, x);
          hi = max(hi, x);
        }
      }
    });
    __syncthreads();   // every warp has read the histogram
    clear();
    (void)team.sum_range(0u, lo, hi);
    __syncthreads();
    kmin = lo;
    kmax = hi;
    linear = false;
  }
}

// The list of one token: the k largest of its n keys in ascending index
// order, looked up in the table, -1 behind them, and the list's cells.
template <int THREADS>
__device__ __forceinline__ void write_list(Team<THREADS>& team, SelScratch& sc, const uint32_t* keys, int n, int k,
                                           const int32_t* table, int32_t* out_blk, int32_t* out_idx,
                                           int32_t* out_len, int bs, int cells) {
  const KeyRun<THREADS> run(keys, n);
  const Threshold th = find_threshold(team, run, k, sc);
  __syncthreads();   // (the bins and the ranked keys are free from here on)
  // keys taken above the threshold and equal to it, before each thread's own
  uint32_t own = 0;
  run.each([&](const uint4& v, int) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t x = c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w;
      own += (x > th.thr ? 0x10000u : 0u) + (x == th.thr && x != 0u ? 1u : 0u);
    }
  });
  if ((int)threadIdx.x == 0) sc.last = 0;
  const uint32_t before = team.before(own);
  __syncthreads();   // (sc.last)
  uint32_t gb = before >> 16, eb = before & 0xffffu;
  // Lists that fit go through shared memory, so their block ids are looked
  // up all at once.
  const bool staged = th.count <= kListMax;
  if (own != 0)
    run.each([&](const uint4& v, int i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t x = c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w;
        const bool above = x > th.thr, equal = x == th.thr && x != 0u;
        if (above || (equal && eb < th.ties)) {
          const uint32_t at = gb + min(eb, th.ties);
          if (staged) {
            sc.list[at] = (uint16_t)(i + c);
          } else {
            out_blk[at] = __ldg(table + i + c);
            if (out_idx != nullptr) out_idx[at] = i + c;
          }
          if (i + c == n - 1) sc.last = 1;
        }
        gb += above;
        eb += equal;
      }
    });
  __syncthreads();
#pragma unroll 4
  for (int i = (int)threadIdx.x; i < k; i += THREADS) {
    if (i < th.count && !staged) continue;
    const int j = i < th.count ? sc.list[i] : -1;
    out_blk[i] = j >= 0 ? __ldg(table + j) : -1;
    if (out_idx != nullptr) out_idx[i] = j;
  }
  if ((int)threadIdx.x == 0) *out_len = th.count * bs - (sc.last ? bs - 1 - (cells - 1) % bs : 0);
}

// The list of one token that takes every block of its row that is the pool's.
template <int THREADS>
__device__ __forceinline__ void take_all(SelScratch& sc, int n, int n_blocks, int k, const int32_t* table,
                                         int32_t* out_blk, int32_t* out_idx, int32_t* out_len, int bs, int cells) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int count = 0;
  bool last = false;
#pragma unroll 1
  for (int j0 = 0; j0 < n; j0 += THREADS) {
    const int j = j0 + tid, blk = j < n ? __ldg(table + j) : -1;
    const unsigned m = __ballot_sync(kAll, (unsigned)blk < (unsigned)n_blocks);
    if (lane == 0) sc.sums[0][0][warp] = (uint32_t)__popc(m);
    last |= __syncthreads_or(j == n - 1 && ((m >> lane) & 1u)) != 0;
    int at = count + __popc(m & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      const int c = (int)sc.sums[0][0][w];
      at += w < warp ? c : 0;
      count += c;
    }
    if ((m >> lane) & 1u) {
      out_blk[at] = blk;
      if (out_idx != nullptr) out_idx[at] = j;
    }
    __syncthreads();   // the counts are written again
  }
#pragma unroll 1
  for (int i = count + tid; i < k; i += THREADS) {
    out_blk[i] = -1;
    if (out_idx != nullptr) out_idx[i] = -1;
  }
  if (tid == 0) *out_len = count * bs - (last ? bs - 1 - (cells - 1) % bs : 0);
}

// NT n-tiles of 8 query rows; THREADS 256 (3 CTAs an SM where the
// registers allow it, else 2) or 512 (one).
template <int HD, int NT, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 1 : NT == 1 && HD <= 128 ? 3 : 2)
    select_blocks_kernel(SelectArgs a) {
  constexpr int kSelWarps = THREADS / 32;
  constexpr int NG = HD / kGroup;
  constexpr int STRIP = 16;               // blocks a warp scores at once
  constexpr int DEPTH = NG < 2 ? NG : 2;  // units (16 blocks x 64 dims) whose loads a warp has in flight
  constexpr int CHAINS = NT <= 2 ? 2 : 1;   // (registers)
  constexpr bool BREG = NT == 1 && HD <= 128 && THREADS == 512;   // q fragments stay in registers
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ SelScratch sc;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t rank = cta_rank();
  const int C = a.cluster;
  cluster_arrive();   // every CTA of the cluster runs before a remote store below
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int bs = 1 << a.bs_log2;
  // this cluster's (sequence, KV head, tokens w0 ..)
  int id = blockIdx.x / C;
  const int wg = id % a.n_wg;
  id /= a.n_wg;
  const int h = id % a.n_kv;
  int b = id / a.n_kv, len_raw;
  if (a.order) {
    // Sequences go by length, longest first, in kOrderSteps steps of max_ctx:
    // clusters start roughly in order, and short rows fill the end of the
    // launch (64 ragged sequences: 79 -> 74 us).
    const int rank_b = b;
    const float step = (float)kOrderSteps / ((float)a.n_cap * (float)bs);
    int v[kOrderRegs], base = 0;
#pragma unroll
    for (int i = 0; i < kOrderRegs; ++i) v[i] = lane + 32 * i < a.n_seq ? __ldg(a.ctx_lens + lane + 32 * i) : 0;
    len_raw = 0;
    bool found = false;
#pragma unroll 1
    for (int c = kOrderSteps - 1; c >= 0 && !found; --c)
#pragma unroll
      for (int i = 0; i < kOrderRegs; ++i) {
        if (32 * i >= a.n_seq || found) continue;
        const int cls = min(max((int)((float)v[i] * step), 0), kOrderSteps - 1);
        const unsigned m = __ballot_sync(kAll, lane + 32 * i < a.n_seq && cls == c);
        const int k = rank_b - base;   // the k-th of them, if it is among these
        if (k < __popc(m)) {
          const unsigned hit = __ballot_sync(kAll, ((m >> lane) & 1u) && __popc(m & ((1u << lane) - 1u)) == k);
          b = 32 * i + __ffs(hit) - 1;
          len_raw = __shfl_sync(kAll, v[i], b & 31);
          found = true;
        }
        base += __popc(m);
      }
  } else {
    len_raw = __ldg(a.ctx_lens + b);
  }
  const int w0 = wg * a.wg_tok, nw = min(a.wg_tok, a.W - w0);
  // the query rows: a warp per (padded row, 64 dims), two dims a lane
  constexpr int QPW = (NT * 8 * NG + kSelWarps - 1) / kSelWarps;
  float2 qv[QPW];
#pragma unroll
  for (int k = 0; k < QPW; ++k) {
    const int i = min(warp + k * kSelWarps, NT * 8 * NG - 1), r = i / NG, gq = i - r * NG;
    const int w = min(r >> a.gp_log2, nw - 1), gg = min(r & ((1 << a.gp_log2) - 1), a.G - 1);
    const float* src = a.q + (((size_t)b * a.W + w0 + w) * a.n_q + (size_t)h * a.G + gg) * HD + gq * kGroup;
    qv[k] = __ldg(reinterpret_cast<const float2*>(src) + lane);
  }
  const long long cap = min((long long)a.max_blocks << a.bs_log2, (long long)a.n_cap << a.bs_log2);
  const int len = (int)max(0LL, min((long long)len_raw, cap));
  auto visible = [&](int w) { return max(0, len - a.W + w0 + w + 1); };        // cells token w0 + w sees
  auto blocks_of = [&](int cells) { return (cells >> a.bs_log2) + ((cells & (bs - 1)) != 0); };
  const int32_t* table = a.block_table + (size_t)b * a.max_blocks;
  const SelSmem lay = sel_smem(HD, NT, a.lead_rows, a.n_cap);
  uint32_t* s_q = reinterpret_cast<uint32_t*>(smem);
  float* s_scale = reinterpret_cast<float*>(smem + lay.scales);
  uint32_t* s_keys = reinterpret_cast<uint32_t*>(smem + lay.keys);

  const int n_all = blocks_of(visible(nw - 1));
  auto out_row = [&](int w) { return ((size_t)b * a.W + w0 + w) * a.n_kv + h; };
  auto index_of = [&](size_t row) { return a.sel_index != nullptr ? a.sel_index + row * a.n_sel : nullptr; };
  if (__builtin_expect(n_all <= a.n_sel, 0)) {
    // What the last token sees, and with it every other, fits the list: all of
    // it is taken without a score (8 heads of 2048 cells, 64 blocks of 64 a
    // list, 4.4 -> 2.2 us; 64 sequences of 100 to 4096 cells 10.6 -> 5.3 us; the
    // branch costs longer rows 1 to 2 %).
    cluster_wait();
    for (int w = (int)rank; w < nw; w += C) {
      const size_t row = out_row(w);
      take_all<THREADS>(sc, blocks_of(visible(w)), a.n_blocks, a.n_sel, table, a.sel_blocks + row * a.n_sel,
                        index_of(row), a.sel_lens + row, bs, visible(w));
    }
    return;
  }

  // this CTA's share of the blocks the last token sees; its first ids are on
  // their way while the q codes are made
  const int share = ((n_all + C - 1) / C + STRIP - 1) / STRIP * STRIP;
  const int j0 = min((int)rank * share, n_all), j1 = min(j0 + share, n_all);
  constexpr int STEP = kSelWarps * STRIP;
  auto load_ids = [&](int s0) -> int {
    return s0 + (lane & 15) < j1 ? __ldg(table + s0 + (lane & 15)) : -1;
  };
  // A lane's loads of group q of a strip: dims 16 t .. + 15 of blocks g and
  // g + 8, lo and hi.  A foreign block reads block 0 (it gets no key).
  struct Unit {
    uint4 lo[2], hi[2];
    float ks[2];
  };
  struct Rows {
    const int8_t* bound[2];
    const float* scale[2];
  };
  auto rows_of = [&](int ids) -> Rows {
    Rows x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int blk = __shfl_sync(kAll, ids, g + 8 * i);
      const size_t row = (size_t)((unsigned)blk < (unsigned)a.n_blocks ? blk : 0) * a.n_kv + h;
      x.bound[i] = a.bounds + row * 2 * HD + t * 16;
      x.scale[i] = a.scales + row * NG;
    }
    return x;
  };
  auto load_unit = [&](const Rows& x, int gq, Unit& u) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u.lo[i] = __ldg(reinterpret_cast<const uint4*>(x.bound[i] + gq * kGroup));
      u.hi[i] = __ldg(reinterpret_cast<const uint4*>(x.bound[i] + gq * kGroup + HD));
      u.ks[i] = __ldg(x.scale[i] + gq);
    }
  };
  const int first = j0 + warp * STRIP;
  int ids = load_ids(first), ids_next = load_ids(first + STEP);

  // q codes
#pragma unroll
  for (int k = 0; k < QPW; ++k) {
    const int i = warp + k * kSelWarps, r = i / NG, gq = i - r * NG;
    if (i >= NT * 8 * NG) break;
    float2 x = qv[k];
    x.x = x.x == x.x ? x.x : 0.f;
    x.y = x.y == x.y ? x.y : 0.f;
    const float m = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(fmaxf(fabsf(x.x), fabsf(x.y)))));
    const int e = q_exponent(m);
    const float inv = pow2f_exact(-e);
    const float c0 = rintf(fminf(fmaxf(x.x * inv, -127.f), 127.f));
    const float c1 = rintf(fminf(fmaxf(x.y * inv, -127.f), 127.f));
    // dims 2 lane, + 1 of the group: fragment lane 4 (r % 8) + lane / 8,
    // k-step (lane % 8) / 2, word lane % 2
    const int at = ((((r >> 3) * NG + gq) * 4 + ((lane & 7) >> 1)) * 2) * 64 + ((r & 7) * 4 + (lane >> 3)) * 2 + (lane & 1);
    s_q[at] = pack_half2(fminf(c0, 0.f), fminf(c1, 0.f));
    s_q[at + 64] = pack_half2(fmaxf(c0, 0.f), fmaxf(c1, 0.f));
    if (lane == 0) s_scale[r * NG + gq] = pow2f_exact(e);
  }
  Unit unit[DEPTH];
  Rows rows = rows_of(ids);
#pragma unroll
  for (int q = 0; q < DEPTH; ++q) load_unit(rows, q, unit[q]);
  __syncthreads();

  const uint32_t keys_addr = static_cast<uint32_t>(__cvta_generic_to_shared(s_keys));
  auto b_frag = [&](int nt, int q, int kk, int which) -> uint2 {
    return *reinterpret_cast<const uint2*>(s_q + (((nt * NG + q) * 4 + kk) * 2 + which) * 64 + lane * 2);
  };
  uint2 breg[BREG ? NG : 1][4][2];
  if constexpr (BREG) {
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int which = 0; which < 2; ++which) breg[q][kk][which] = b_frag(0, q, kk, which);
  }
  const int gp = 1 << a.gp_log2;
  // The tokens whose keys this lane writes, from column c = 0 (and, one row a
  // token, 1) of each n-tile: the blocks they see (0: not this lane's to
  // write) and where their keys go.
  constexpr int TOKS = 2;
  int tok_nb[NT][TOKS];
  uint32_t tok_at[NT][TOKS];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < TOKS; ++c) {
      const int row = nt * 8 + 2 * t + c, w = row >> a.gp_log2, lead_row = w >> a.c_log2;
      // (more than 8 rows a token: written at its last n-tile)
      const bool mine = gp <= 8 ? (row & (gp - 1)) == 0 : t == 0 && c == 0 && ((nt * 8 + 8) & (gp - 1)) == 0;
      tok_nb[nt][c] = mine && w < nw ? blocks_of(visible(w)) : 0;
      const uint32_t at = keys_addr + (uint32_t)(lead_row * key_row(a.n_cap)) * 4u;
      asm("mapa.shared::cluster.u32 %0, %1, %2;"
          : "=r"(tok_at[nt][c])
          : "r"(at), "r"((uint32_t)(w - (lead_row << a.c_log2)) & (uint32_t)(C - 1)));
    }
  auto emit = [&](int nt, int c, int j, bool valid, float best) {
    const int nb = tok_nb[nt][c];
    if (nb == 0 || j >= j1) return;
    uint32_t key = 0;
    if (j < nb && valid) key = (j < a.n_first || j >= nb - a.n_last) ? kForced : ordered(best);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(tok_at[nt][c] + 4u * (uint32_t)j), "r"(key) : "memory");
  };

  __syncwarp();
  cluster_wait();
  for (int s0 = first; s0 < j1; s0 += STEP) {
    const int ids_cur = ids;
    ids = ids_next;
    ids_next = load_ids(s0 + 2 * STEP);
    const Rows rows_cur = rows;
    rows = rows_of(ids);
    float z[NT][4], z2[NG == 4 ? NT : 1][4];   // score sums: blocks g (0, 1), g + 8 (2, 3), rows 2t, 2t + 1
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      Unit& u = unit[q % DEPTH];
      float acc[NT][CHAINS][4];   // lo and hi sums apart: shorter chains (whole numbers both)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4 * CHAINS; ++k) acc[nt][k >> 2][k & 3] = 0.f;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        // fp16 fragments of the group: k-step kk is the lane's word kk
        uint32_t af[4][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 v = which ? u.hi[i] : u.lo[i];
          widen(v.x, af[0][i], af[0][2 + i]);
          widen(v.y, af[1][i], af[1][2 + i]);
          widen(v.z, af[2][i], af[2][2 + i]);
          widen(v.w, af[3][i], af[3][2 + i]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            uint2 bf;
            if constexpr (BREG) bf = breg[q][kk][which];
            else bf = b_frag(nt, q, kk, which);
            mma_f16(acc[nt][which % CHAINS], af[kk], bf.x, bf.y);
          }
      }
      const float ks0 = u.ks[0], ks1 = u.ks[1];
      // the unit DEPTH further on, of this strip or the next
      if (q + DEPTH < NG) load_unit(rows_cur, q + DEPTH, u);
      else load_unit(rows, q + DEPTH - NG, u);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float qs = s_scale[(nt * 8 + 2 * t + c) * NG + q];
          // S * (scale_q * scale_k), both exact; groups add pairwise
#pragma unroll
          for (int k = c; k < 4; k += 2) {
            const float v = __fmul_rn(CHAINS == 2 ? acc[nt][0][k] + acc[nt][CHAINS - 1][k] : acc[nt][0][k], __fmul_rn(qs, k < 2 ? ks0 : ks1));
            if (q == 0) z[nt][k] = v;
            else if (q == 1) z[nt][k] = __fadd_rn(z[nt][k], v);
            else if (q == 2) z2[NG == 4 ? nt : 0][k] = v;
            else z[nt][k] = __fadd_rn(z[nt][k], __fadd_rn(z2[NG == 4 ? nt : 0][k], v));
          }
        }
    }
    // the largest over a token's rows, then its keys
    const bool va = (unsigned)__shfl_sync(kAll, ids_cur, g) < (unsigned)a.n_blocks;
    const bool vb = (unsigned)__shfl_sync(kAll, ids_cur, g + 8) < (unsigned)a.n_blocks;
    const int ja = s0 + g, jb = s0 + g + 8;
    if (gp == 1) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          emit(nt, c, ja, va, z[nt][c]);
          emit(nt, c, jb, vb, z[nt][2 + c]);
        }
    } else {
      float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m0 = fmaxf(m0, fmaxf(z[nt][0], z[nt][1]));
        m1 = fmaxf(m1, fmaxf(z[nt][2], z[nt][3]));
        if (gp > 8 && ((nt * 8 + 8) & (gp - 1)) != 0) continue;   // (the token goes on)
        if (gp >= 4) {
          m0 = fmaxf(m0, __shfl_xor_sync(kAll, m0, 1));
          m1 = fmaxf(m1, __shfl_xor_sync(kAll, m1, 1));
        }
        if (gp >= 8) {
          m0 = fmaxf(m0, __shfl_xor_sync(kAll, m0, 2));
          m1 = fmaxf(m1, __shfl_xor_sync(kAll, m1, 2));
        }
        emit(nt, 0, ja, va, m0);
        emit(nt, 0, jb, vb, m1);
        m0 = m1 = -INFINITY;
      }
    }
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();   // every key is in its leader's shared memory

  // ---------------- selection: token w is led by CTA w % C ----------------
  auto keys_of = [&](int w) { return s_keys + (size_t)(w >> a.c_log2) * key_row(a.n_cap); };
  Team<THREADS> team{sc};
  for (int w = (int)rank; w < nw; w += C) {
    const size_t row = out_row(w);
    write_list(team, sc, keys_of(w), blocks_of(visible(w)), a.n_sel, table, a.sel_blocks + row * a.n_sel,
               index_of(row), a.sel_lens + row, bs, visible(w));
    if (w + C < nw) __syncthreads();   // the scratch is reused by the next token
  }
}

template <int HD, int NT, int THREADS>
cudaError_t launch_nt(const SelectArgs& a, cudaStream_t s) {
  static ContextCache<int> cache;
  int ready = 0;
  if (!per_context(cache, &ready, [](int* v) {
        *v = 1;
        // clusters of 16 are past the portable 8
        return cudaFuncSetAttribute(select_blocks_kernel<HD, NT, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSelMaxSmem) == cudaSuccess &&
               cudaFuncSetAttribute(select_blocks_kernel<HD, NT, THREADS>,
                                    cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
      }))
    return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  const long long ctas = (long long)a.n_seq * a.n_kv * a.n_wg * a.cluster;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = sel_smem(HD, NT, a.lead_rows, a.n_cap).bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_blocks_kernel<HD, NT, THREADS>, a);
}

int n_tiles(const SelectArgs& a) {
  const int rows = a.wg_tok << a.gp_log2;
  return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}

template <int HD>
cudaError_t launch_hd(const SelectArgs& a, cudaStream_t s) {
  const int nt = n_tiles(a);
  if (a.wide) {
    if (nt == 1) return launch_nt<HD, 1, 512>(a, s);
    if (nt == 2) return launch_nt<HD, 2, 512>(a, s);
    return launch_nt<HD, 4, 512>(a, s);
  }
  if (nt == 1) return launch_nt<HD, 1, 256>(a, s);
  if (nt == 2) return launch_nt<HD, 2, 256>(a, s);
  return launch_nt<HD, 4, 256>(a, s);
}

}  // namespace

bool plan_select(int hd, int sms, SelectArgs* a) {
  a->gp_log2 = 0;
  while ((1 << a->gp_log2) < a->G) ++a->gp_log2;
  // tokens per cluster: up to 32 padded rows, for which the bounds are read
  // once
  const int max_tok = 32 >> a->gp_log2;
  a->wg_tok = a->W < max_tok ? a->W : max_tok;
  for (;;) {
    a->n_wg = (a->W + a->wg_tok - 1) / a->wg_tok;
    const long long clusters = (long long)a->n_seq * a->n_kv * a->n_wg;
    // CTAs per cluster: as many as fill the SMs once, at least 64 blocks each
    // and at most 8 (16 from 8192 blocks: 16384 blocks x 2 heads 29 us, with
    // 8 CTAs 42 us; 512 blocks x 8 heads 6.1 us either way, 4096 blocks x 8
    // heads x 4 tokens 15.6 us, with 8 CTAs 12.7 us); for batches of longer rows
    // up to four times the SMs, at least 512 blocks each (64 sequences of up
    // to 4096 blocks 73 -> 68 us; 32 sequences of up to 2048 blocks, 4 tokens,
    // 35 us, with 1024 blocks each 44 us, with 256 43 us).
    const int most = a->n_cap >= 8192 ? 4 : 3;
    int c = 0;
    while (c < most && (clusters << c) < sms && a->n_cap >= (64 << c)) ++c;
    while (c < most && (clusters << c) < 4 * sms && a->n_cap >= (1024 << c)) ++c;
    a->c_log2 = c;
    a->cluster = 1 << c;
    a->order = a->n_seq > 1 && a->n_seq <= 32 * kOrderRegs && (clusters << c) > 2 * sms;
    // 512 threads where rows are long and the CTAs take half of the SMs at
    // most (4096 blocks x 8 heads x 4 tokens 14.6 -> 12.7 us, 16384 x 2 40 -> 29
    // us; 4096 x 16, on 128 CTAs, 14.4 us with 256 threads, 16.4 with 512)
    a->wide = a->n_cap >= 2048 && (clusters << c) * 2 <= sms;
    a->lead_rows = (a->wg_tok + a->cluster - 1) >> c;
    const bool fits = sel_smem(hd, n_tiles(*a), a->lead_rows, a->n_cap).bytes <= kSelMaxSmem;
    // Where that leaves more than half of the SMs idle, fewer tokens a cluster
    // (their bounds are then read again, from L2): 4096 blocks x 2 heads x 256
    // dims x 4 tokens 19.5 -> 12.9 us, 256 blocks x 8 heads x 4 tokens 6.5 ->
    // 6.2.  Long rows stop sooner, at two fifths of the SMs, because their
    // clusters have to find places together.  On 64 CTAs and on 128, blocks x
    // heads x tokens: 2048 x 8 x 4 9.5 and 10.1 us, 3000 x 8 x 4 11.5 and 12.5,
    // 4096 x 8 x 4 12.7 and 15.0 (64 dims 11.3 and 13.1, 256 dims 15.1 and
    // 18.9), 6000 x 8 x 4 15.4 and 19.0, 4096 x 8 x 2 11.6 and 14.9, 4096 x 4 x
    // 8 12.7 and 15.1, 12000 x 4 x 4 18.5 and 27.1.
    const bool fills = (clusters << c) * 2 > sms || (a->n_cap >= 2048 && (clusters << c) * 5 > 2 * sms);
    if (fits && (fills || a->wg_tok == 1)) return true;
    if (a->wg_tok == 1) return false;
    a->wg_tok = (a->wg_tok + 1) / 2;
  }
}

cudaError_t launch_select_blocks(int hd, const SelectArgs& a, cudaStream_t s) {
  if (hd == 64) return launch_hd<64>(a, s);
  if (hd == 128) return launch_hd<128>(a, s);
  return launch_hd<256>(a, s);
}

}  // namespace kvq
