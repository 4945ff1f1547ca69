// kvq_select.cu -- the blocks each query token and KV head attends to
// (kvq_select_blocks): a score for every block from its key bounds, and the
// n_sel highest.
//
// The score bounds q . k over a block's keys from above: per dim the larger
// of q lo and q hi, i.e. max(q, 0) hi + min(q, 0) lo.  q enters as int8
// codes with a power-of-two scale per 64 dims, the bounds are int8 codes
// with a power-of-two scale per 64 dims, so a group's sum S is a whole
// number below 2^21 and S * scale_q * scale_k is exact in fp32; 2 or 4
// groups are added pairwise in fp32, and the query heads of a KV head give
// their maximum.  No sum depends on its order, so the chosen blocks do not
// depend on how the work is split; ties go to the lower block.
//
// One cluster of CTAs per (sequence, KV head, up to kMaxTok tokens).  The
// CTAs share the visible blocks: each lane holds 16 dims of a block (one
// 16-byte load of lo and of hi), the q codes of 4 query heads in registers,
// and sums by dp4a (4 products an instruction); the lanes of a group meet by
// shuffles.  Each key (the score as an order-preserving integer) goes
// straight to the shared memory of the CTA that leads its token's selection
// (distributed shared memory).  After one cluster barrier the leaders find
// the n_sel-th largest key by radix counting from the first bit in which the
// keys differ, and write the list in ascending order.
#include <math.h>
#include <stdint.h>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kDigitBits = 10;
constexpr int kBins = 1 << kDigitBits;
constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kForced = 0xffffffffu;   // keys: 0 not a candidate, kForced always kept

// The smallest e with 127 * 2^e >= m (m >= 0, finite or inf), in [-60, 60].
__device__ __forceinline__ int q_exponent(float m) {
  const uint32_t b = __float_as_uint(m);
  const int e = (int)(b >> 23) - 126 - 7 + ((b & 0x7fffffu) > 0x7e0000u);
  return min(max(e, -60), 60);
}

__device__ __forceinline__ float pow2f_exact(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// fp32 (no NaN) -> uint32 in the same order; finite scores map inside
// (0x007fffff, 0xff800000), clear of 0 and kForced.  -0 counts as +0.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void store_remote(uint32_t addr, uint32_t rank, uint32_t v) {
  asm volatile(
      "{\n .reg .b32 ra;\n mapa.shared::cluster.u32 ra, %0, %1;\n st.shared::cluster.u32 [ra], %2;\n}\n" ::"r"(addr),
      "r"(rank), "r"(v)
      : "memory");
}

// Layout of the dynamic shared memory.
struct SelSmem {
  int codes, scales, keys, bytes;
};
__host__ __device__ inline SelSmem sel_smem(int hd, int rows, int lead_rows, int n_cap) {
  SelSmem m;
  m.codes = 0;                                   // [rows][2][hd] int8: min(c, 0), max(c, 0)
  m.scales = rows * 2 * hd;                      // [rows][hd / 64] fp32
  m.keys = (m.scales + rows * (hd / kGroup) * 4 + 15) / 16 * 16;   // [lead_rows][n_cap] uint32
  m.bytes = m.keys + lead_rows * n_cap * 4;
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

__device__ Threshold find_threshold(const uint32_t* keys, int n, int k, uint32_t* s_hist, uint32_t* s_aux) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // counts of candidates and forced ones, range of the others
  uint32_t cand = 0, forced = 0, kmin = 0xffffffffu, kmax = 0;
  for (int i = tid; i < n; i += kSelThreads) {
    const uint32_t x = keys[i];
    cand += x != 0;
    forced += x == kForced;
    if (x != 0 && x != kForced) {
      kmin = min(kmin, x);
      kmax = max(kmax, x);
    }
  }
  cand = __reduce_add_sync(kAll, cand);
  forced = __reduce_add_sync(kAll, forced);
  kmin = __reduce_min_sync(kAll, kmin);
  kmax = __reduce_max_sync(kAll, kmax);
  if (lane == 0) {
    s_aux[warp] = cand;
    s_aux[kSelWarps + warp] = forced;
    s_aux[2 * kSelWarps + warp] = kmin;
    s_aux[3 * kSelWarps + warp] = kmax;
  }
  for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
  __syncthreads();
  cand = forced = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    cand += s_aux[w];
    forced += s_aux[kSelWarps + w];
    kmin = min(kmin, s_aux[2 * kSelWarps + w]);
    kmax = max(kmax, s_aux[3 * kSelWarps + w]);
  }
  if ((int)cand <= k) return {0u, 0u, (int)cand};                   // all of them
  if ((int)forced >= k) return {kForced, (uint32_t)k, k};           // (forced <= k by the call's checks)
  uint32_t rem = (uint32_t)k - forced;                              // 1 <= rem < others
  int bits = kmin == kmax ? 0 : 32 - __clz(kmin ^ kmax);            // the keys differ below this bit
  uint32_t base = bits >= 32 ? 0u : kmin & ~((1u << bits) - 1u);
  while (bits > 0) {
    const int d = min(bits, kDigitBits), shift = bits - d;
    const uint32_t mask = (1u << d) - 1u;
    // keys that share the bits above this digit (>> 1 first: bits may be 32)
    const uint32_t top = (base >> 1) >> (bits - 1);
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t x = keys[i];
      if (x != 0 && x != kForced && ((x >> 1) >> (bits - 1)) == top) atomicAdd(&s_hist[(x >> shift) & mask], 1u);
    }
    __syncthreads();
    // thread t: bins kBins - 1 - 4t .. kBins - 4 - 4t (from the top down)
    constexpr int BPT = kBins / kSelThreads;
    uint32_t c[BPT], sum = 0;
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
      c[j] = s_hist[kBins - 1 - (tid * BPT + j)];
      sum += c[j];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_aux[warp] = incl;
    __syncthreads();
    uint32_t above = incl - sum;
    for (int w = 0; w < warp; ++w) above += s_aux[w];
    if (above < rem && above + sum >= rem) {   // exactly one thread
#pragma unroll
      for (int j = 0; j < BPT; ++j) {
        if (above < rem && above + c[j] >= rem) {
          s_aux[kSelWarps] = (uint32_t)(kBins - 1 - (tid * BPT + j));
          s_aux[kSelWarps + 1] = rem - above;
          s_aux[kSelWarps + 2] = c[j];
        }
        above += c[j];
      }
    }
    // (the histogram is read: clear it for the next digit)
#pragma unroll
    for (int j = 0; j < BPT; ++j) s_hist[kBins - 1 - (tid * BPT + j)] = 0;
    __syncthreads();
    base |= s_aux[kSelWarps] << shift;
    rem = s_aux[kSelWarps + 1];
    const uint32_t in_bin = s_aux[kSelWarps + 2];
    bits = shift;
    if (in_bin == rem) return {base == 0 ? 0u : base - 1u, 0u, k};   // the bin is taken whole
  }
  return {base, rem, k};
}

// RC query heads of one token are scored together.
template <int HD, int RC>
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(SelectArgs a) {
  constexpr int LPB = HD / 16;            // lanes per block
  constexpr int BPP = 32 / LPB;           // blocks per warp pass
  constexpr int NG = HD / kGroup;
  constexpr int PASSES = HD == 256 ? 4 : 2;
  constexpr int STRIP = BPP * PASSES;     // blocks whose loads a warp has in flight: 16, 8, 8
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint32_t s_hist[kBins];
  __shared__ uint32_t s_aux[4 * kSelWarps + 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cta_rank();
  const int C = a.cluster;
  cluster_arrive();   // every CTA of the cluster runs before a remote store below
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // this cluster's (sequence, KV head, tokens w0 ..)
  int id = blockIdx.x / C;
  const int wg = id % a.n_wg;
  id /= a.n_wg;
  const int h = id % a.n_kv, b = id / a.n_kv;
  const int w0 = wg * a.wg_tok, nw = min(a.wg_tok, a.W - w0);
  const long long cap = min((long long)a.max_blocks << a.bs_log2, (long long)a.n_cap << a.bs_log2);
  const int len = (int)max(0LL, min((long long)__ldg(a.ctx_lens + b), cap));
  const int bs = 1 << a.bs_log2;
  auto visible = [&](int w) { return max(0, len - a.W + w0 + w + 1); };        // cells token w0 + w sees
  auto blocks_of = [&](int cells) { return (cells + bs - 1) >> a.bs_log2; };
  const int32_t* table = a.block_table + (size_t)b * a.max_blocks;
  const int rows = nw * a.G;
  const SelSmem lay = sel_smem(HD, a.wg_tok * a.G, a.lead_rows, a.n_cap);
  int8_t* s_codes = reinterpret_cast<int8_t*>(smem + lay.codes);
  float* s_scale = reinterpret_cast<float*>(smem + lay.scales);
  uint32_t* s_keys = reinterpret_cast<uint32_t*>(smem + lay.keys);

  // q codes: a warp per (row, 64 dims), two dims a lane
  for (int i = warp; i < rows * NG; i += kSelWarps) {
    const int r = i / NG, g = i - r * NG;
    const int w = r / a.G, gg = r - w * a.G;
    const float* src = a.q + (((size_t)b * a.W + w0 + w) * a.n_q + (size_t)h * a.G + gg) * HD + g * kGroup;
    float2 x = __ldg(reinterpret_cast<const float2*>(src) + lane);
    x.x = x.x == x.x ? x.x : 0.f;
    x.y = x.y == x.y ? x.y : 0.f;
    const float m = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(fmaxf(fabsf(x.x), fabsf(x.y)))));
    const int e = q_exponent(m);
    const float inv = pow2f_exact(-e);
    const int c0 = __float2int_rn(fminf(fmaxf(x.x * inv, -127.f), 127.f));
    const int c1 = __float2int_rn(fminf(fmaxf(x.y * inv, -127.f), 127.f));
    char2* neg = reinterpret_cast<char2*>(s_codes + (size_t)r * 2 * HD + g * kGroup) + lane;
    char2* pos = reinterpret_cast<char2*>(s_codes + (size_t)r * 2 * HD + HD + g * kGroup) + lane;
    *neg = make_char2((signed char)min(c0, 0), (signed char)min(c1, 0));
    *pos = make_char2((signed char)max(c0, 0), (signed char)max(c1, 0));
    if (lane == 0) s_scale[r * NG + g] = pow2f_exact(e);
  }
  __syncthreads();

  // this CTA's share of the blocks the last token sees
  const int n_all = blocks_of(visible(nw - 1));
  const int share = ((n_all + C - 1) / C + STRIP - 1) / STRIP * STRIP;
  const int j0 = min((int)rank * share, n_all), j1 = min(j0 + share, n_all);
  const int l = lane % LPB, sub = lane / LPB;      // lane's dims 16 l .. + 15 of block sub of a pass
  const uint32_t keys_addr = static_cast<uint32_t>(__cvta_generic_to_shared(s_keys));
  const int n_chunks = (a.G + RC - 1) / RC;

  // q codes (min and max parts) and scales of RC heads, the lane's dims; a
  // chunk past the group's end repeats its last head, which leaves the
  // maximum over heads as it is
  auto load_q = [&](int w, int ch, uint4 (&qn)[RC], uint4 (&qp)[RC], float (&qs)[RC]) {
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      const int r = w * a.G + min(ch * RC + i, a.G - 1);
      const int8_t* base = s_codes + (size_t)r * 2 * HD + l * 16;
      qn[i] = *reinterpret_cast<const uint4*>(base);
      qp[i] = *reinterpret_cast<const uint4*>(base + HD);
      qs[i] = s_scale[r * NG + l / 4];
    }
  };
  // this lane's score of one row chunk: which of the RC rows it holds after
  // the reduction does not matter, the caller takes the maximum over them
  auto score = [&](const uint4& lo, const uint4& hi, float ks, const uint4 (&qn)[RC], const uint4 (&qp)[RC],
                   const float (&qs)[RC]) -> float {
    int s[RC];
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      int v = __dp4a((int)lo.x, (int)qn[i].x, 0);
      v = __dp4a((int)hi.x, (int)qp[i].x, v);
      v = __dp4a((int)lo.y, (int)qn[i].y, v);
      v = __dp4a((int)hi.y, (int)qp[i].y, v);
      v = __dp4a((int)lo.z, (int)qn[i].z, v);
      v = __dp4a((int)hi.z, (int)qp[i].z, v);
      v = __dp4a((int)lo.w, (int)qn[i].w, v);
      s[i] = __dp4a((int)hi.w, (int)qp[i].w, v);
    }
    // sum over the 4 lanes of the 64 dims; with 4 rows each lane ends with
    // one row's sum, with 2 rows each pair of lanes
    int v;
    float sc;
    if constexpr (RC == 4) {
      const bool odd = lane & 1, two = lane & 2;
      const int k0 = odd ? s[2] : s[0], k1 = odd ? s[3] : s[1];
      const int g0 = odd ? s[0] : s[2], g1 = odd ? s[1] : s[3];
      const int a0 = k0 + __shfl_xor_sync(kAll, g0, 1), a1 = k1 + __shfl_xor_sync(kAll, g1, 1);
      v = (two ? a1 : a0) + __shfl_xor_sync(kAll, two ? a0 : a1, 2);
      sc = odd ? (two ? qs[3] : qs[2]) : (two ? qs[1] : qs[0]);
    } else if constexpr (RC == 2) {
      const bool odd = lane & 1;
      v = (odd ? s[1] : s[0]) + __shfl_xor_sync(kAll, odd ? s[0] : s[1], 1);
      v += __shfl_xor_sync(kAll, v, 2);
      sc = odd ? qs[1] : qs[0];
    } else {
      v = s[0] + __shfl_xor_sync(kAll, s[0], 1);
      v += __shfl_xor_sync(kAll, v, 2);
      sc = qs[0];
    }
    float t = (float)v * (sc * ks);
    if constexpr (NG >= 2) t += __shfl_xor_sync(kAll, t, 4);
    if constexpr (NG >= 4) t += __shfl_xor_sync(kAll, t, 8);
    return t;
  };
  auto emit = [&](int w, int j, int blk, float best) {
    const int nb = blocks_of(visible(w));
    uint32_t key = 0;
    if (j < nb && blk >= 0 && blk < a.n_blocks)
      key = (j < a.n_first || j >= nb - a.n_last) ? kForced : ordered(best);
    const uint32_t lead = (uint32_t)w % (uint32_t)C, row = (uint32_t)w / (uint32_t)C;
    store_remote(keys_addr + (row * (uint32_t)a.n_cap + (uint32_t)j) * 4u, lead, key);
  };

  uint4 qn[RC], qp[RC];
  float qs[RC];
  const bool fixed_q = nw == 1 && n_chunks == 1;   // one chunk: q stays in registers
  if (fixed_q) load_q(0, 0, qn, qp, qs);
  __syncwarp();
  cluster_wait();
  for (int s0 = j0 + warp * STRIP; s0 < j1; s0 += kSelWarps * STRIP) {
    // physical ids of the strip, then every bound of it
    const int my = s0 + lane < j1 && lane < STRIP ? __ldg(table + s0 + lane) : -1;
    uint4 lo[PASSES], hi[PASSES];
    float ks[PASSES];
    int blk[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      blk[p] = __shfl_sync(kAll, my, p * BPP + sub);
      lo[p] = hi[p] = make_uint4(0, 0, 0, 0);
      ks[p] = 0.f;
      if (blk[p] >= 0 && blk[p] < a.n_blocks) {
        const size_t row = (size_t)blk[p] * a.n_kv + h;
        const int8_t* src = a.bounds + row * 2 * HD + l * 16;
        lo[p] = __ldg(reinterpret_cast<const uint4*>(src));
        hi[p] = __ldg(reinterpret_cast<const uint4*>(src + HD));
        ks[p] = __ldg(a.scales + row * NG + l / 4);
      }
    }
    for (int w = 0; w < nw; ++w) {
      float best[PASSES];
#pragma unroll
      for (int p = 0; p < PASSES; ++p) best[p] = -INFINITY;
      for (int ch = 0; ch < n_chunks; ++ch) {
        if (!fixed_q) load_q(w, ch, qn, qp, qs);
#pragma unroll
        for (int p = 0; p < PASSES; ++p) best[p] = fmaxf(best[p], score(lo[p], hi[p], ks[p], qn, qp, qs));
      }
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        float v = best[p];
        if constexpr (RC >= 2) v = fmaxf(v, __shfl_xor_sync(kAll, v, 1));
        if constexpr (RC >= 4) v = fmaxf(v, __shfl_xor_sync(kAll, v, 2));
        const int j = s0 + p * BPP + sub;
        if (l == 0 && j < j1) emit(w, j, blk[p], v);
      }
    }
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();   // every key is in its leader's shared memory

  // ---------------- selection: token w is led by CTA w % C ----------------
  for (int w = (int)rank; w < nw; w += C) {
    const uint32_t* keys = s_keys + (size_t)(w / C) * a.n_cap;
    const int cells = visible(w), nb = blocks_of(cells);
    const size_t out_row = ((size_t)b * a.W + w0 + w) * a.n_kv + h;
    int32_t* out_blk = a.sel_blocks + out_row * a.n_sel;
    int32_t* out_idx = a.sel_index != nullptr ? a.sel_index + out_row * a.n_sel : nullptr;
    const Threshold th = find_threshold(keys, nb, a.n_sel, s_hist, s_aux);
    // each warp lists a contiguous range of blocks
    const int seg = ((nb + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int i0 = min(warp * seg, nb), i1 = min(i0 + seg, nb);
    int gt = 0, eq = 0;
    for (int i = i0; i < i1; i += 32) {
      const uint32_t x = i + lane < i1 ? keys[i + lane] : 0u;
      gt += __popc(__ballot_sync(kAll, x > th.thr));
      eq += __popc(__ballot_sync(kAll, x == th.thr && x != 0u));
    }
    __syncthreads();   // s_aux is free again
    if (lane == 0) {
      s_aux[warp] = (uint32_t)gt;
      s_aux[kSelWarps + warp] = (uint32_t)eq;
    }
    if (tid == 0) s_aux[2 * kSelWarps] = 0;
    __syncthreads();
    uint32_t gb = 0, eb = 0;   // taken above, and equal, in the ranges before
    for (int v = 0; v < warp; ++v) {
      gb += s_aux[v];
      eb += s_aux[kSelWarps + v];
    }
    const uint32_t lt = (1u << lane) - 1u;
    for (int i = i0; i < i1; i += 32) {
      const uint32_t x = i + lane < i1 ? keys[i + lane] : 0u;
      const uint32_t mg = __ballot_sync(kAll, x > th.thr), me = __ballot_sync(kAll, x == th.thr && x != 0u);
      const uint32_t ebl = eb + __popc(me & lt);
      const bool take = ((mg >> lane) & 1u) || (((me >> lane) & 1u) && ebl < th.ties);
      if (take) {
        const uint32_t at = gb + __popc(mg & lt) + min(ebl, th.ties);
        out_blk[at] = __ldg(table + i + lane);
        if (out_idx != nullptr) out_idx[at] = i + lane;
        if (i + lane == nb - 1) s_aux[2 * kSelWarps] = 1u;
      }
      gb += __popc(mg);
      eb += __popc(me);
    }
    for (int i = th.count + tid; i < a.n_sel; i += kSelThreads) {
      out_blk[i] = -1;
      if (out_idx != nullptr) out_idx[i] = -1;
    }
    __syncthreads();
    if (tid == 0) a.sel_lens[out_row] = th.count * bs - (s_aux[2 * kSelWarps] ? nb * bs - cells : 0);
    __syncthreads();   // s_aux and the histogram are reused by the next token
  }
}

template <int HD, int RC>
cudaError_t launch_rc(const SelectArgs& a, cudaStream_t s) {
  static ContextCache<int> cache;
  int ready = 0;
  if (!per_context(cache, &ready, [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(select_blocks_kernel<HD, RC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSelMaxSmem) == cudaSuccess;
      }))
    return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  const long long ctas = (long long)a.n_seq * a.n_kv * a.n_wg * a.cluster;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = sel_smem(HD, a.wg_tok * a.G, a.lead_rows, a.n_cap).bytes;
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
  return cudaLaunchKernelEx(&cfg, select_blocks_kernel<HD, RC>, a);
}

template <int HD>
cudaError_t launch_hd(const SelectArgs& a, cudaStream_t s) {
  if (a.G == 1) return launch_rc<HD, 1>(a, s);
  if (a.G == 2) return launch_rc<HD, 2>(a, s);
  return launch_rc<HD, 4>(a, s);
}

}  // namespace

bool plan_select(int hd, int sms, SelectArgs* a) {
  // tokens per cluster: as many as keep the q codes at 32 rows, whose
  // bounds are then read once
  const int max_tok = 32 / a->G;
  a->wg_tok = a->W < max_tok ? a->W : max_tok;
  // CTAs per cluster: enough to fill the SMs, at least 64 blocks each
  int c = 1;
  for (;;) {
    a->n_wg = (a->W + a->wg_tok - 1) / a->wg_tok;
    const long long clusters = (long long)a->n_seq * a->n_kv * a->n_wg;
    c = 1;
    while (c < 8 && clusters * c < sms && a->n_cap >= 128 * c) c *= 2;
    a->cluster = c;
    a->lead_rows = (a->wg_tok + c - 1) / c;
    if (sel_smem(hd, a->wg_tok * a->G, a->lead_rows, a->n_cap).bytes <= kSelMaxSmem) return true;
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
