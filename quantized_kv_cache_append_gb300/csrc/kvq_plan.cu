// kvq_plan.cu -- block tables and slot maps of one serving step, built on
// the GPU from the requests' lengths (kvq_plan_step).
//
// Sequence b holds ceil(ctx_in[b] / block_size) blocks.  With n_new[b] >= 0
// it grows to ceil((ctx_in[b] + n_new[b]) / block_size); with n_new[b] < 0
// it ends and gives its blocks back.  Three exclusive prefix sums over the
// sequences (tokens, blocks handed out, blocks given back) place everything:
//
//   given back  j = 0 .. P-1   row entries of the released sequences, in
//                              (sequence, column) order, pushed on the stack
//   handed out  i = 0 .. A-1   popped off its top, to the growing sequences
//                              in (sequence, column) order: pushed[P - 1 - i]
//                              while i < P, then free_list[count - 1 - (i - P)]
//   token       t = 0 .. T-1   its sequence by a binary search in the token
//                              prefix, its position, and its cell
//
// One launch, no workspace: every CTA computes the prefixes of all sequences
// into its own shared memory (a few KB read from L2) and then writes its
// share of the tokens, table entries and list entries.  Nothing one CTA
// writes is read by another: new table entries lie past the old ones, a
// given-back block is either handed out again or stored above the old stack
// top by the thread that reads it, pops below the old top read entries nobody
// writes, and the lengths and the count are not updated in place (the call
// refuses overlapping arrays).
#include <stdint.h>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

// 256 threads and 2 CTAs an SM: 700 sequences with 1,000,003 tokens 10.1 us, 64
// sequences with a token each 4.1 us (512 x 1: 10.1, 4.4; 1024 x 1: 10.9, 5.7).
constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanPerSm = 2;
constexpr int kPlanSeqPerCta = 128;   // at least one CTA for so many sequences (16384: 30 -> 21 us)
constexpr unsigned kFullMask = 0xffffffffu;

// The three sums, held at kMost (lengths come from the device and may be
// anything; no step that can be placed comes near it, so what is held there
// is refused).
constexpr uint32_t kMost = (1u << 30) + 1u;
struct Three {
  uint32_t tok, grow, back;
};

__device__ __forceinline__ Three operator+(const Three& a, const Three& b) {
  return {min(a.tok + b.tok, kMost), min(a.grow + b.grow, kMost), min(a.back + b.back, kMost)};
}

__device__ __forceinline__ Three shfl_up(const Three& a, int d) {
  return {__shfl_up_sync(kFullMask, a.tok, d), __shfl_up_sync(kFullMask, a.grow, d),
          __shfl_up_sync(kFullMask, a.back, d)};
}

// What one sequence adds to the three sums; bad: it does not fit its row of
// the table.
__device__ __forceinline__ Three of_sequence(const PlanArgs& a, int ctx, int n, bool& bad) {
  const long long end = (long long)ctx + max(n, 0);
  bad |= ctx < 0 || end > (long long)a.max_blocks << a.bs_log2;
  if (ctx < 0) return {0, 0, 0};
  const uint32_t up = (1u << a.bs_log2) - 1u, have = ((uint32_t)ctx + up) >> a.bs_log2;   // (< 2^32)
  if (n < 0) return {0, 0, have};
  return {min((uint32_t)n, kMost), (uint32_t)((end + up) >> a.bs_log2) - have, 0};
}

// First sequence whose inclusive prefix end[] is above x (x < end[n - 1]).
__device__ __forceinline__ int owner_of(const uint32_t* end, int n, uint32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_step_kernel(PlanArgs a) {
  // inclusive prefixes over the sequences, shifted by one: end[b] at [b + 1]
  extern __shared__ uint32_t s_pref[];
  const int n = a.n_seq;
  uint32_t* s_tok = s_pref;
  uint32_t* s_grow = s_pref + (n + 1);
  uint32_t* s_back = s_pref + 2 * (n + 1);
  __shared__ uint4 s_warp[kPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Each thread sums a run of consecutive sequences, the runs are scanned.
  // Longer runs than 4 take their lengths through shared memory, where the
  // prefixes replace them: read in whole lines, and of odd length, so the
  // threads' runs start in different banks (16384 sequences 76 -> 31 us).
  const long long count = __ldg(a.free_count_in);
  const bool staged = n > 4 * kPlanThreads;
  int per = (n + kPlanThreads - 1) / kPlanThreads;
  if (staged) {
#pragma unroll 4
    for (int b = tid; b < n; b += kPlanThreads) {
      s_tok[b + 1] = (uint32_t)__ldg(a.ctx_in + b);
      s_grow[b + 1] = (uint32_t)__ldg(a.n_new + b);
    }
    __syncthreads();
    per |= 1;
  }
  const int b0 = min(tid * per, n), b1 = min(b0 + per, n);
  auto of = [&](int b, bool& bad) -> Three {
    return staged ? of_sequence(a, (int)s_tok[b + 1], (int)s_grow[b + 1], bad)
                  : of_sequence(a, __ldg(a.ctx_in + b), __ldg(a.n_new + b), bad);
  };
  Three sum = {0, 0, 0};
  bool bad = false;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) sum = sum + of(b, bad);
  Three incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Three y = shfl_up(incl, d);
    if (lane >= d) incl = incl + y;
  }
  if (lane == 31) s_warp[warp] = make_uint4(incl.tok, incl.grow, incl.back, 0);
  const bool any_bad = __syncthreads_or(bad);
  Three base = {0, 0, 0}, total = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    const uint4 v = s_warp[w];
    if (w < warp) base = base + Three{v.x, v.y, v.z};
    total = total + Three{v.x, v.y, v.z};
  }
  int status = 0;
  if (total.tok > (uint32_t)a.max_tok) status |= KVQ_PLAN_TOKENS;
  if (any_bad) status |= KVQ_PLAN_ROW;
  if ((long long)total.grow > count + (long long)total.back) status |= KVQ_PLAN_BLOCKS;
  if (count < 0 || count + (long long)total.back > a.n_blocks) status |= KVQ_PLAN_LIST;
  const bool ok = status == 0;
  const int gtid = blockIdx.x * kPlanThreads + tid, gthreads = gridDim.x * kPlanThreads;

  if (!ok) {  // nothing changes: the lengths stay, no token is placed
    for (int b = gtid; b < n; b += gthreads) a.ctx_out[b] = __ldg(a.ctx_in + b);
    for (int b = gtid; b < n + 1; b += gthreads) a.tok_start[b] = 0;
    for (int t = gtid; t < a.max_tok; t += gthreads) {
      a.tok_seq[t] = -1;
      a.tok_pos[t] = -1;
      if (a.slots != nullptr) a.slots[t] = -1;
    }
    if (gtid == 0) {
      *a.free_count_out = (int32_t)count;
      *reinterpret_cast<int4*>(a.info) = make_int4(0, 0, 0, status);
    }
    return;
  }

  // (no sum is held from here on)
  Three run = base + incl;
  run = {run.tok - sum.tok, run.grow - sum.grow, run.back - sum.back};
  if (tid == 0) s_tok[0] = s_grow[0] = s_back[0] = 0;
  bool unused = false;
  for (int b = b0; b < b1; ++b) {
    run = run + of(b, unused);
    s_tok[b + 1] = run.tok;
    s_grow[b + 1] = run.grow;
    s_back[b + 1] = run.back;
  }
  __syncthreads();
  const uint32_t T = total.tok, A = total.grow, P = total.back;
  const int bs_mask = (1 << a.bs_log2) - 1;

  auto pushed = [&](uint32_t j) -> int32_t {   // j-th block given back
    const int b = owner_of(s_back + 1, n, j);
    return __ldg(a.block_table + (size_t)b * a.max_blocks + (j - s_back[b]));
  };
  auto handed = [&](uint32_t i) -> int32_t {   // i-th block handed out
    return i < P ? pushed(P - 1 - i) : __ldg(a.free_list + ((uint32_t)count - 1 - (i - P)));
  };

  // lengths, token starts, totals
  for (int b = gtid; b < n + 1; b += gthreads) {
    a.tok_start[b] = (int32_t)s_tok[b];
    if (b < n) {
      const int nn = __ldg(a.n_new + b);
      a.ctx_out[b] = nn < 0 ? 0 : __ldg(a.ctx_in + b) + nn;
    }
  }
  if (gtid == 0) {
    *a.free_count_out = (int32_t)((uint32_t)count + P - A);
    *reinterpret_cast<int4*>(a.info) = make_int4((int)T, (int)A, (int)P, 0);
  }
  // the new table entries, and what stays on the stack above its old top
  for (uint32_t i = gtid; i < A; i += gthreads) {
    const int b = owner_of(s_grow + 1, n, i);
    const int have = (__ldg(a.ctx_in + b) + bs_mask) >> a.bs_log2;
    a.block_table_out[(size_t)b * a.max_blocks + have + (i - s_grow[b])] = handed(i);
  }
  if (P > A)
    for (uint32_t j = gtid; j < P - A; j += gthreads) a.free_list_out[(uint32_t)count + j] = pushed(j);

  // tokens: 4 consecutive ones a thread, one search, then a walk; a block is
  // looked up once for the tokens that share it
  for (long long t4 = 4LL * gtid; t4 < a.max_tok; t4 += 4LL * gthreads) {
    int32_t seq[4], pos[4], slot[4];
    int b = t4 < T ? owner_of(s_tok + 1, n, (uint32_t)t4) : 0;
    int col = -1, blk = -1, ctx = 0, have = 0;
    uint32_t t0 = 0, t1 = 0;   // the sequence's tokens
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long t = t4 + u;
      seq[u] = pos[u] = slot[u] = -1;
      if (t < T) {
        if ((uint32_t)t >= t1) {
          while (s_tok[b + 1] <= (uint32_t)t) ++b;
          t0 = s_tok[b];
          t1 = s_tok[b + 1];
          ctx = __ldg(a.ctx_in + b);
          have = (ctx + bs_mask) >> a.bs_log2;
          col = -1;
        }
        seq[u] = b;
        pos[u] = ctx + (int)((uint32_t)t - t0);
        if (a.slots != nullptr) {
          const int c = pos[u] >> a.bs_log2;
          if (c != col) {
            col = c;
            blk = c < have ? __ldg(a.block_table + (size_t)b * a.max_blocks + c)
                           : handed(s_grow[b] + (uint32_t)(c - have));
          }
          slot[u] = (blk << a.bs_log2) | (pos[u] & bs_mask);
        }
      }
    }
    if (t4 + 4 <= a.max_tok) {
      *reinterpret_cast<int4*>(a.tok_seq + t4) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      *reinterpret_cast<int4*>(a.tok_pos + t4) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (a.slots != nullptr)
        *reinterpret_cast<int4*>(a.slots + t4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t4 + u < a.max_tok) {
          a.tok_seq[t4 + u] = seq[u];
          a.tok_pos[t4 + u] = pos[u];
          if (a.slots != nullptr) a.slots[t4 + u] = slot[u];
        }
    }
  }
}

}  // namespace

cudaError_t launch_plan_step(const PlanArgs& a, int sms, cudaStream_t s) {
  static ContextCache<int> cache;
  int ready = 0;
  if (!per_context(cache, &ready, [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(plan_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    plan_smem_bytes(kPlanMaxSeq)) == cudaSuccess;
      }))
    return cudaErrorInvalidConfiguration;
  const long long per_cta = 4LL * kPlanThreads;
  long long ctas = (a.max_tok + per_cta - 1) / per_cta;
  // (released sequences give back far more blocks than tokens come in)
  const long long by_seq = (a.n_seq + kPlanSeqPerCta - 1) / kPlanSeqPerCta;
  if (ctas < by_seq) ctas = by_seq;
  if (ctas > kPlanPerSm * sms) ctas = kPlanPerSm * sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = plan_smem_bytes(a.n_seq);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_step_kernel, a);
}

}  // namespace kvq
