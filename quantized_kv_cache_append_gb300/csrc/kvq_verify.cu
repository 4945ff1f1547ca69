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
// A cluster of CTAs shares a row, tile by tile of 512 or 1024 values: each warp
// keeps its tiles' sums in shared memory, the CTAs send each other their
// totals, the one that holds the place finds the tile and reads it once more
// (from L2).  Rows start at any element (a vocabulary is rarely a multiple of
// 16 bytes): the tiles count from the 16-byte boundary before the target's
// row, and the draft's values are shifted into place out of two 16-byte loads
// (the second from L1).
#include <cuda_bf16.h>

#include "kvq_internal.cuh"
#include "kvq_ptx.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace {

constexpr int kVerThreads = 256;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kGranules = 4;   // 16-byte loads of a row a lane has in flight: a tile
template <class E>
constexpr int kTile = kGranules * 32 * 16 / (int)sizeof(E);
constexpr int kMostCtas = 8;
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

// value e of a granule
template <class E>
__device__ __forceinline__ float value(const uint4& g, int e) {
  const uint32_t w[4] = {g.x, g.y, g.z, g.w};
  if constexpr (sizeof(E) == 4) return __uint_as_float(w[e]);
  else if constexpr (sizeof(E) == 2 && !__is_same(E, __half))
    return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
  else return e & 1 ? half_hi(w[e >> 1]) : half_lo(w[e >> 1]);
}

// A sum of weights in whole numbers: floor(r * 2^40) = h * 2^20 + l for r in
// [0, 1].  Adding 2^23 with rounding down leaves the whole part in the low
// mantissa bits, everything else is exact; the exponent bits that come along
// are taken off once (sums mod 2^32: a tile's values keep h and l below 2^31).
struct Count {
  uint32_t h, l;
};
constexpr uint32_t kMagicBits = 0x4b000000u;   // 2^23

__device__ __forceinline__ void add_weight(Count& c, float r) {
  constexpr float k20 = 1048576.0f, k23 = 8388608.0f;
  const float a = __fmaf_rd(r, k20, k23);
  const float rest = __fmaf_rn(r, k20, k23 - a);
  c.h += __float_as_uint(a);
  c.l += __float_as_uint(__fmaf_rd(rest, k20, k23));
}
__device__ __forceinline__ unsigned long long total_of(const Count& c, int n) {   // n values in it
  return ((unsigned long long)(c.h - (uint32_t)n * kMagicBits) << 20) + (c.l - (uint32_t)n * kMagicBits);
}

// The row that is sampled: weights p, p - q, or p without one token, held in
// [0, 1] (NaN: 0).  Places count from `pad` values before the row, where the
// target's address is a multiple of 16; weights there and behind the row
// are 0.  [p_lo, p_hi) and [q_lo, q_hi) are the whole arrays.
template <class E>
struct Row {
  const E* p;      // of place 0
  const E* q;      // of place 0, or null
  int without;     // a place, or -1
  int pad, end;    // the row: places [pad, end)
  const char *p_lo, *p_hi, *q_lo, *q_hi;
};

// The 16 bytes that start 4 WORDS + bits / 8 bytes into v0 | v1.
template <int WORDS>
__device__ __forceinline__ uint4 shifted(const uint4& v0, const uint4& v1, int bits) {
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  return make_uint4(__funnelshift_r(w[WORDS], w[WORDS + 1], bits), __funnelshift_r(w[WORDS + 1], w[WORDS + 2], bits),
                    __funnelshift_r(w[WORDS + 2], w[WORDS + 3], bits),
                    __funnelshift_r(w[WORDS + 3], w[WORDS + 4], bits));
}

// Bytes p + 512 k + 0 .. 15, k < kGranules; the granules that hold them are
// all in the array.
__device__ __forceinline__ void load_tile(const char* p, uint4 (&v)[kGranules]) {
  const int s = (int)(reinterpret_cast<uintptr_t>(p) & 15);   // (the same in all lanes)
  const uint4* g = reinterpret_cast<const uint4*>(p - s);
#pragma unroll
  for (int k = 0; k < kGranules; ++k) v[k] = __ldg(g + 32 * k);
  if (s != 0) {
    uint4 n[kGranules];
    const int bits = 8 * (s & 3);
#pragma unroll
    for (int k = 0; k < kGranules; ++k) n[k] = __ldg(g + 32 * k + 1);
    switch (s >> 2) {
      case 0:
#pragma unroll
        for (int k = 0; k < kGranules; ++k) v[k] = shifted<0>(v[k], n[k], bits);
        break;
      case 1:
#pragma unroll
        for (int k = 0; k < kGranules; ++k) v[k] = shifted<1>(v[k], n[k], bits);
        break;
      case 2:
#pragma unroll
        for (int k = 0; k < kGranules; ++k) v[k] = shifted<2>(v[k], n[k], bits);
        break;
      default:
#pragma unroll
        for (int k = 0; k < kGranules; ++k) v[k] = shifted<3>(v[k], n[k], bits);
    }
  }
}

// Whether a tile's granules lie in the array (t: its first byte).
__device__ __forceinline__ bool inside(const char* t, const char* lo, const char* hi) {
  const int s = (int)(reinterpret_cast<uintptr_t>(t) & 15);
  return t - s >= lo && t - s + 512 * kGranules + (s != 0 ? 16 : 0) <= hi;
}

// A lane's weights of a tile: r[k NV + e] is that of place (32 k + lane) NV + e
// of it.
template <class E>
__device__ __forceinline__ void tile_weights(const Row<E>& row, int tile, int lane, float (&r)[kTile<E> / 32]) {
  constexpr int NV = 16 / (int)sizeof(E);
  const int i0 = tile * kTile<E>, at0 = i0 + lane * NV;
  const char *tp = reinterpret_cast<const char*>(row.p + i0), *tq = reinterpret_cast<const char*>(row.q + i0);
  const bool has_q = row.q != nullptr;
  if (inside(tp, row.p_lo, row.p_hi) && (!has_q || inside(tq, row.q_lo, row.q_hi))) {
    uint4 p[kGranules], q[kGranules];
    load_tile(tp + 16 * lane, p);
    if (has_q) {
      load_tile(tq + 16 * lane, q);
#pragma unroll
      for (int k = 0; k < kGranules; ++k)
#pragma unroll
        for (int e = 0; e < NV; ++e) r[k * NV + e] = __saturatef(value<E>(p[k], e) - value<E>(q[k], e));
    } else {
#pragma unroll
      for (int k = 0; k < kGranules; ++k)
#pragma unroll
        for (int e = 0; e < NV; ++e) r[k * NV + e] = __saturatef(value<E>(p[k], e));
    }
  } else {   // at an array's ends, value by value
#pragma unroll
    for (int k = 0; k < kGranules; ++k)
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        const int i = at0 + 32 * NV * k + e;
        const bool in = i >= row.pad && i < row.end;
        float x = in ? wide(row.p[i]) : 0.f;
        if (in && has_q) x -= wide(row.q[i]);
        r[k * NV + e] = __saturatef(x);
      }
  }
  // the places outside the row, and the one left out: in few tiles
  if (i0 < row.pad || i0 + kTile<E> > row.end || (unsigned)(row.without - i0) < (unsigned)kTile<E>) {
#pragma unroll
    for (int k = 0; k < kGranules; ++k)
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        const int i = at0 + 32 * NV * k + e;
        if (i < row.pad || i >= row.end || i == row.without) r[k * NV + e] = 0.f;
      }
  }
}

// The same for two weights, in packed instructions (7 instead of 12).
__device__ __forceinline__ void add_weights(Count& c, float r0, float r1) {
  uint32_t h0, h1, l0, l1;
  asm("{\n"
      " .reg .b64 r, k20, k23, one, a, d, e;\n"
      " mov.b64 r, {%4, %5};\n"
      " mov.b64 k20, {%6, %6};\n"
      " mov.b64 k23, {%7, %7};\n"
      " mov.b64 one, {%8, %8};\n"
      " fma.rm.f32x2 a, r, k20, k23;\n"
      " fma.rn.f32x2 d, a, one, k23;\n"     // k23 - a
      " fma.rn.f32x2 d, r, k20, d;\n"
      " fma.rm.f32x2 e, d, k20, k23;\n"
      " mov.b64 {%0, %1}, a;\n"
      " mov.b64 {%2, %3}, e;\n"
      "}"
      : "=r"(h0), "=r"(h1), "=r"(l0), "=r"(l1)
      : "f"(r0), "f"(r1), "f"(1048576.0f), "f"(8388608.0f), "f"(-1.0f));
  c.h += h0 + h1;
  c.l += l0 + l1;
}

template <int N>
__device__ __forceinline__ Count count_of(const float* r) {
  Count c = {0, 0};
#pragma unroll
  for (int e = 0; e < N; e += 2) add_weights(c, r[e], r[e + 1]);
  return c;
}

__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long y = __shfl_up_sync(kFullMask, v, d);
    if (lane >= d) v += y;
  }
  return v;
}

__device__ __forceinline__ void st_dsmem_u64(uint32_t addr, int rank, unsigned long long v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote), "l"(v) : "memory");
}

// 4 CTAs an SM: 256 sequences of 131075 bf16 tokens 23.6 us (2 or 3 CTAs 32 us, 5
// 31 us; half tiles 28 to 39 us; weights one by one 24.5; twice as many CTAs a row
// 27.5).
template <int T>
__global__ void __launch_bounds__(kVerThreads, 4) verify_kernel(const __grid_constant__ VerifyArgs a) {
  using E = typename Prob<T>::type;
  constexpr int NV = 16 / (int)sizeof(E), N = kGranules;
  __shared__ unsigned long long s_tile[(1 << 20) / kTile<E> + 1];
  __shared__ unsigned long long s_total[2][kMostCtas];   // [residual, row][CTA], sent by each of them
  __shared__ int s_a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n_cta = 1 << a.c_log2;
  const int b = blockIdx.x >> a.c_log2, rank = blockIdx.x & (n_cta - 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = a.W;
  const E* target = static_cast<const E*>(a.target);
  const E* draft = static_cast<const E*>(a.draft);
  // the small loads together: lane i of every warp looks at draft i
  const int n_raw = a.n_draft != nullptr ? __ldg(a.n_draft + b) : W - 1;
  const float us = __ldg(a.u_sample + b);
  int x = -1;
  float u = 0.f;
  if (lane < W - 1) {
    x = __ldg(a.draft_tokens + (size_t)b * (W - 1) + lane);
    u = __ldg(a.u + (size_t)b * (W - 1) + lane);
  }
  const int n_given = min(n_raw, W - 1);
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
  // (waited for before the first store into a peer's shared memory: all of the
  // cluster's CTAs run by then)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  // how many drafts stand
  if (warp == 0) {
    bool ok = false;
    if (lane < W - 1 && x >= 0 && x < a.vocab) {
      const float p = wide(target[((long long)b * W + lane) * a.target_stride + x]);
      const float q =
          draft != nullptr ? wide(draft[((long long)b * (W - 1) + lane) * a.draft_stride + x]) : 1.0f;
      ok = lane < n_given && (double)u * (double)q < (double)p;
    }
    const unsigned no = __ballot_sync(kFullMask, !ok);   // (lane 31 never is: W <= 32)
    if (lane == 0) s_a = __ffs(no) - 1;
  }
  __syncthreads();
  const int n_acc = s_a;
  const bool rejected = n_acc < n_given;
  Row<E> row;
  const E* first = target + ((long long)b * W + n_acc) * a.target_stride;
  row.pad = (int)((reinterpret_cast<uintptr_t>(first) & 15) / sizeof(E));
  row.end = row.pad + a.vocab;
  row.p = first - row.pad;
  row.q = rejected && draft != nullptr ? draft + ((long long)b * (W - 1) + n_acc) * a.draft_stride - row.pad : nullptr;
  row.without = __shfl_sync(kFullMask, x, n_acc);
  row.without = rejected && draft == nullptr && row.without >= 0 && row.without < a.vocab ? row.without + row.pad : -1;
  row.p_lo = static_cast<const char*>(a.target);
  row.p_hi = reinterpret_cast<const char*>(target + ((long long)a.n_seq * W - 1) * a.target_stride + a.vocab);
  row.q_lo = static_cast<const char*>(a.draft);
  row.q_hi = reinterpret_cast<const char*>(draft + ((long long)a.n_seq * (W - 1) - 1) * a.draft_stride + a.vocab);

  const int tiles = (row.end + kTile<E> - 1) / kTile<E>, per = (tiles + n_cta - 1) >> a.c_log2;
  const int t0 = min(rank * per, tiles), n_mine = min(t0 + per, tiles) - t0;
  unsigned long long S = 0, before = 0, mine = 0;
  for (int pass = 0; pass < 2; ++pass) {
    for (int t = warp; t < n_mine; t += kVerWarps) {
      float r[kTile<E> / 32];
      tile_weights<E>(row, t0 + t, lane, r);
      Count c = count_of<kTile<E> / 32>(r);
      c.h = __reduce_add_sync(kFullMask, c.h);
      c.l = __reduce_add_sync(kFullMask, c.l);
      if (lane == 0) s_tile[t] = total_of(c, kTile<E>);
    }
    __syncthreads();
    if (pass == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) {
      unsigned long long v = 0;
      for (int t = lane; t < n_mine; t += 32) v += s_tile[t];
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
      if (lane < n_cta) st_dsmem_u64(smem_u32(&s_total[pass][rank]), lane, v);
    }
    cluster_sync_all();   // (a CTA's shared memory is written by its peers before this only)
    S = before = 0;
    for (int r = 0; r < n_cta; ++r) {
      const unsigned long long v = s_total[pass][r];
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
  const unsigned long long U =
      (unsigned long long)fminf(fmaxf(us * 16777216.0f, 0.0f), 16777215.0f);   // (truncates; NaN: 0)
  const unsigned long long mark = (S >> 24) * U + (((S & 0xffffffu) * U) >> 24);
  if (rank == 0 && warp == 0) {
    if (lane < W && (lane != n_acc || S == 0)) tokens[lane] = lane < n_acc ? x : -1;
    if (lane == 0) {
      a.n_accepted[b] = n_acc;
      if (a.n_dropped != nullptr) a.n_dropped[b] = n_given - n_acc;
    }
  }
  if (warp == 0 && S != 0 && mark >= before && mark - before < mine) {
    // the tile that holds the place, its granules' row, the lane, the value
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
    float r[kTile<E> / 32];
    tile_weights<E>(row, t0 + t, lane, r);
    Count c[N];
    int at = -1;
#pragma unroll
    for (int k = 0; k < N; ++k) c[k] = count_of<NV>(r + k * NV);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const Count all = {__reduce_add_sync(kFullMask, c[k].h), __reduce_add_sync(kFullMask, c[k].l)};
      const unsigned long long sum = total_of(all, 32 * NV);
      if (at < 0 && sum > left) {   // (the same in all lanes)
        const unsigned long long v = total_of(c[k], NV);
        const unsigned long long incl = warp_scan(v, lane);
        const int src = __ffs(__ballot_sync(kFullMask, incl > left)) - 1;
        if (lane == src) {
          left -= incl - v;
          bool found = false;
#pragma unroll
          for (int e = 0; e < NV; ++e) {
            Count one = {0, 0};
            add_weight(one, r[k * NV + e]);
            const unsigned long long w = total_of(one, 1);
            if (!found && w > left) {
              found = true;
              tokens[n_acc] = (t0 + t) * kTile<E> + (32 * k + lane) * NV + e - row.pad;
            }
            if (!found) left -= w;
          }
        }
        at = k;
      }
      if (at < 0) left -= sum;
    }
  }
}

template <int T>
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
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

}  // namespace

cudaError_t launch_verify_draft(int type, VerifyArgs a, int sms, cudaStream_t s) {
  // CTAs of a row: as many as fill the SMs, each with a tile at least
  a.c_log2 = 0;
  const int tiles = (a.vocab + 1023) / 1024;
  while ((2 << a.c_log2) <= kMostCtas && ((long long)a.n_seq << a.c_log2) < 2LL * sms && (2 << a.c_log2) <= tiles)
    ++a.c_log2;
  switch (type) {
    case KVQ_T_F32: return launch<KVQ_T_F32>(a, s);
    case KVQ_T_F16: return launch<KVQ_T_F16>(a, s);
    case KVQ_T_BF16: return launch<KVQ_T_BF16>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
