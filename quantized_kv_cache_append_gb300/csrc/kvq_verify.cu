// kvq_verify.cu -- drafted tokens against the target's probabilities
// (kvq_verify_draft): rejection sampling from given random numbers.
//
//   accept draft i while  u_i * q_i(x_i) < p_i(x_i)             (exact in fp64)
//   then sample from      max(p_a - q_a, 0), or p_a               (a accepted)
//
// One row of p (and of q) per sequence is all that has to be read: HBM or,
// for few sequences, latency bounds it.  Sampling by the inverse of the
// cumulated weights needs their sum before the place, so the weights are
// whole numbers, floor(r * 2^40): their sums do not depend on the order, the
// answer does not depend on how the row is split, and it equals the
// definition's bit for bit.
//
// A cluster of CTAs shares a row, tile by tile of 1024 values: each warp
// keeps its tiles' sums in shared memory, the CTAs exchange their totals, the
// one that holds the place finds the tile and reads it once more (from L2).
#include <cuda_bf16.h>

#include "kvq_internal.cuh"
#include "kvq_ptx.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace {

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kTile = 1024;
constexpr int kMostTiles = (1 << 20) / kTile;
constexpr unsigned kFullMask = 0xffffffffu;

template <int T>
struct Prob;
template <>
struct Prob<KVQ_T_F32> {
  using type = float;
};
template <>
struct Prob<KVQ_T_F16> {
  using type = __half;
};
template <>
struct Prob<KVQ_T_BF16> {
  using type = __nv_bfloat16;
};

__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ float wide(__half x) { return __half2float(x); }
__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }

// floor(min(max(r, 0), 1) * 2^40) = h * 2^20 + l: adding 2^23 with rounding
// down leaves the whole part in the mantissa, everything else is exact.
// (fmaxf takes 0 for NaN.)
__device__ __forceinline__ void add_units(float r, uint32_t& h, uint32_t& l) {
  const float x = fminf(fmaxf(r, 0.0f), 1.0f) * 1048576.0f;
  const float a = __fadd_rd(x, 8388608.0f);
  const float b = __fadd_rd((x - (a - 8388608.0f)) * 1048576.0f, 8388608.0f);
  h += __float_as_uint(a) & 0x7fffffu;
  l += __float_as_uint(b) & 0x7fffffu;
}

__device__ __forceinline__ unsigned long long units(float r) {
  uint32_t h = 0, l = 0;
  add_units(r, h, l);
  return ((unsigned long long)h << 20) + l;
}

// The row that is sampled: weights p, p - q, or p without one token.
template <class E>
struct Row {
  const E* p;
  const E* q;      // or null
  int without;     // -1: none
  int vocab;

  __device__ __forceinline__ float weight(int i) const {
    const float x = wide(p[i]);
    return q != nullptr ? x - wide(q[i]) : i == without ? 0.0f : x;
  }
};

// VEC values of a 16-byte load each (rows 16-byte aligned); VEC 1: scalar.
template <class E, int VEC>
__device__ __forceinline__ unsigned long long tile_sum(const Row<E>& row, int tile, int lane) {
  constexpr int N = kTile / 32 / VEC;   // loads a lane
  uint32_t h = 0, l = 0;
  const int i0 = tile * kTile + lane * VEC;
  if ((tile + 1) * kTile <= row.vocab) {
    if constexpr (VEC > 1) {
      uint4 pw[N];
#pragma unroll
      for (int k = 0; k < N; ++k) pw[k] = __ldg(reinterpret_cast<const uint4*>(row.p + i0 + 32 * VEC * k));
      if (row.q != nullptr) {
        uint4 qw[N];
#pragma unroll
        for (int k = 0; k < N; ++k) qw[k] = __ldg(reinterpret_cast<const uint4*>(row.q + i0 + 32 * VEC * k));
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            add_units(wide(reinterpret_cast<const E*>(&pw[k])[e]) - wide(reinterpret_cast<const E*>(&qw[k])[e]), h, l);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            add_units(i0 + 32 * VEC * k + e == row.without ? 0.0f : wide(reinterpret_cast<const E*>(&pw[k])[e]), h, l);
      }
    } else {
#pragma unroll 16
      for (int k = 0; k < N; ++k) add_units(row.weight(i0 + 32 * k), h, l);
    }
  } else {
    for (int k = 0; k < N; ++k)
      for (int e = 0; e < VEC; ++e) {
        const int i = i0 + 32 * VEC * k + e;
        if (i < row.vocab) add_units(row.weight(i), h, l);
      }
  }
  // 1024 values: h and l stay below 2^31
  return ((unsigned long long)__reduce_add_sync(kFullMask, h) << 20) + __reduce_add_sync(kFullMask, l);
}

__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long y = __shfl_up_sync(kFullMask, v, d);
    if (lane >= d) v += y;
  }
  return v;
}

__device__ __forceinline__ unsigned long long ld_dsmem_u64(uint32_t addr, int rank) {
  uint32_t remote;
  unsigned long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote) : "memory");
  return v;
}

template <int T, bool VEC>
__global__ void __launch_bounds__(kVerThreads) verify_kernel(const __grid_constant__ VerifyArgs a) {
  using E = typename Prob<T>::type;
  __shared__ unsigned long long s_tile[kMostTiles];
  __shared__ unsigned long long s_total[2];   // of this CTA: the residual's, the row's
  __shared__ int s_a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n_cta = 1 << a.c_log2;
  const int b = blockIdx.x >> a.c_log2, rank = blockIdx.x & (n_cta - 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = a.W;
  const E* target = static_cast<const E*>(a.target);
  const E* draft = static_cast<const E*>(a.draft);
  const int n_given = a.n_draft != nullptr ? min(__ldg(a.n_draft + b), W - 1) : W - 1;
  int* tokens = a.tokens + (size_t)b * W;
  if (n_given < 0) {   // takes no part (the same in every CTA of the cluster)
    if (rank == 0) {
      if (tid < W) tokens[tid] = -1;
      if (tid == 0) {
        a.n_accepted[b] = 0;
        if (a.n_dropped != nullptr) a.n_dropped[b] = 0;
      }
    }
    return;
  }
  // how many drafts stand: lane i of warp 0 looks at draft i
  if (warp == 0) {
    bool ok = false;
    if (lane < n_given) {
      const int x = __ldg(a.draft_tokens + (size_t)b * (W - 1) + lane);
      if (x >= 0 && x < a.vocab) {
        const float p = wide(target[((long long)b * W + lane) * a.target_stride + x]);
        const float q =
            draft != nullptr ? wide(draft[((long long)b * (W - 1) + lane) * a.draft_stride + x]) : 1.0f;
        ok = (double)__ldg(a.u + (size_t)b * (W - 1) + lane) * (double)q < (double)p;
      }
    }
    const unsigned no = __ballot_sync(kFullMask, !ok);
    const int n = no != 0 ? __ffs(no) - 1 : 32;
    if (lane == 0) s_a = n;
  }
  __syncthreads();
  const int n_acc = s_a;
  const bool rejected = n_acc < n_given;
  Row<E> row;
  row.p = target + ((long long)b * W + n_acc) * a.target_stride;
  row.q = rejected && draft != nullptr ? draft + ((long long)b * (W - 1) + n_acc) * a.draft_stride : nullptr;
  row.without = rejected && draft == nullptr ? __ldg(a.draft_tokens + (size_t)b * (W - 1) + n_acc) : -1;
  row.vocab = a.vocab;

  const int tiles = (a.vocab + kTile - 1) / kTile, per = (tiles + n_cta - 1) >> a.c_log2;
  const int t0 = min(rank * per, tiles), n_mine = min(t0 + per, tiles) - t0;
  const uint32_t total_addr = smem_u32(s_total);
  unsigned long long S = 0, before = 0, mine = 0;
  for (int pass = 0; pass < 2; ++pass) {
    for (int t = warp; t < n_mine; t += kVerWarps) {
      const unsigned long long v = tile_sum<E, VEC ? 16 / (int)sizeof(E) : 1>(row, t0 + t, lane);
      if (lane == 0) s_tile[t] = v;
    }
    __syncthreads();
    if (warp == 0) {
      unsigned long long v = 0;
      for (int t = lane; t < n_mine; t += 32) v += s_tile[t];
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
      if (lane == 0) s_total[pass] = v;
    }
    cluster_sync_all();
    S = before = 0;
    for (int r = 0; r < n_cta; ++r) {
      const unsigned long long v = ld_dsmem_u64(total_addr + 8 * pass, r);
      if (r < rank) before += v;
      if (r == rank) mine = v;
      S += v;
    }
    // nothing above 0 in the difference: the target's own row (every CTA of the
    // cluster sees the same sum)
    if (S != 0 || !rejected || pass == 1) break;
    row.q = nullptr;
    row.without = -1;
  }
  const float us = __ldg(a.u_sample + b);
  const unsigned long long U =
      (unsigned long long)fminf(fmaxf(us * 16777216.0f, 0.0f), 16777215.0f);   // (truncates; NaN: 0)
  const unsigned long long mark = (S >> 24) * U + (((S & 0xffffffu) * U) >> 24);
  if (rank == 0) {
    if (tid < W && (tid != n_acc || S == 0))
      tokens[tid] = tid < n_acc ? __ldg(a.draft_tokens + (size_t)b * (W - 1) + tid) : -1;
    if (tid == 0) {
      a.n_accepted[b] = n_acc;
      if (a.n_dropped != nullptr) a.n_dropped[b] = n_given - n_acc;
    }
  }
  if (warp == 0 && S != 0 && mark >= before && mark - before < mine) {
    // the tile that holds the place, then the value in it
    unsigned long long left = mark - before;   // counts to pass before the place
    int t = 0;
    for (int c = 0; c < n_mine; c += 32) {
      const unsigned long long v = c + lane < n_mine ? s_tile[c + lane] : 0;
      const unsigned long long incl = warp_scan(v, lane);
      const unsigned hit = __ballot_sync(kFullMask, incl > left);
      if (hit != 0) {
        const int src = __ffs(hit) - 1;
        left -= __shfl_sync(kFullMask, incl - v, src);
        t = c + src;
        break;
      }
      left -= __shfl_sync(kFullMask, incl, 31);
    }
    constexpr int N = kTile / 32;
    const int i0 = (t0 + t) * kTile + lane * N;
    unsigned long long sum = 0;
#pragma unroll 8
    for (int k = 0; k < N; ++k) sum += i0 + k < a.vocab ? units(row.weight(i0 + k)) : 0;
    const unsigned long long incl = warp_scan(sum, lane);
    const unsigned hit = __ballot_sync(kFullMask, incl > left);
    if (hit != 0 && lane == __ffs(hit) - 1) {
      left -= incl - sum;
      int i = i0;
      for (; i < i0 + N - 1; ++i) {
        const unsigned long long w = units(row.weight(i));
        if (w > left) break;
        left -= w;
      }
      tokens[n_acc] = i;
    }
  }
  cluster_sync_all();   // no CTA leaves while a peer reads its totals
}

template <int T, bool VEC>
cudaError_t launch(const VerifyArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.n_seq << a.c_log2);
  cfg.blockDim = dim3(kVerThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1u << a.c_log2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, VEC>, a);
}

template <int T>
cudaError_t launch_type(const VerifyArgs& a, cudaStream_t s) {
  constexpr int E = T == KVQ_T_F32 ? 4 : 2;
  const bool vec = (reinterpret_cast<uintptr_t>(a.target) | reinterpret_cast<uintptr_t>(a.draft) |
                    (uintptr_t)(a.target_stride * E) | (uintptr_t)(a.draft != nullptr ? a.draft_stride * E : 0)) %
                       16 == 0;
  return vec ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

}  // namespace

cudaError_t launch_verify_draft(int type, VerifyArgs a, int sms, cudaStream_t s) {
  // CTAs of a row: as many as fill the SMs, each with a tile at least
  a.c_log2 = 0;
  const int tiles = (a.vocab + kTile - 1) / kTile;
  while (a.c_log2 < 3 && ((long long)a.n_seq << a.c_log2) < 2LL * sms && (2 << a.c_log2) <= tiles) ++a.c_log2;
  switch (type) {
    case KVQ_T_F32: return launch_type<KVQ_T_F32>(a, s);
    case KVQ_T_F16: return launch_type<KVQ_T_F16>(a, s);
    case KVQ_T_BF16: return launch_type<KVQ_T_BF16>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
