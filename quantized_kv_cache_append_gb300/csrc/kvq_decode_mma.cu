// kvq_decode_mma.cu -- split-K decode attention on tensor cores, fed by TMA.
//
// The partial kernel of the split-K decode (#3084 qwen35: FP16 K/V cache by
// default, int8 with --kv-q8, "What changed" and "Extra Notes": k_attn_part
// templated on the cache format, read by the decode of the next token).  One
// CTA of 4 warps per (split, KV head, sequence):
//
//   copies      the split's cells stream through a ring of STAGES
//               shared-memory stages of 64 cells: K and V codes by TMA
//               tensor copies (cp.async.bulk.tensor, 128-byte swizzle,
//               straight from the paged pool through the block table), the
//               scales by bulk copies; an mbarrier per stage counts the
//               bytes in.  Thread 0 issues the first stages; after that the
//               warp that releases a stage last (a shared-memory counter)
//               issues its refill (scored: or each warp its own, kWarpSlices).
//   q.k         each warp owns 16 cells of every stage.  S^T = K . Q^T is a
//               16-cell x 8-row mma.sync.m16n8k16 per 16 dims.  int8 K
//               enters as the exact fp16 value 1152 + code, and 1152 * sum(q)
//               per 64-dim group is taken off through the accumulator's
//               starting value; the per-64-dim scales multiply the group
//               partial dot products.
//   softmax     online, in the log2 domain, with a lazily raised reference
//               maximum.
//   p.v         O^T += V^T . P^T, another m16n8k16 per 16 dims; int8 V is
//               widened to fp16 exactly in registers and the V scales are
//               folded into P per group.  K8V4 (#711 kv: --kv k8v4 streams
//               with --kv-resident, "What"): K as int8; V's 4-bit codes
//               widen exactly to code - 8, its per-32 scales fold into P,
//               and each split's merged partial is rotated back
//               (Walsh-Hadamard, / HD) before it is written.
//
// q and p enter the tensor cores as fp16 hi + lo pairs (about 22 significant
// bits), K and V as exact fp16 values.  The copies carry an evict-first L2
// policy: the cache is read once per call.
//
// The CTA's 4 warps merge their states through shared memory into one
// partial (o, m, l) per row of the split; the combine kernel below merges
// the partials of every split.  Masked cells (beyond the context, beyond the causal limit of a
// verify-window row, or in a block whose id is out of range) get logit -inf
// and contribute exact zeros.  Every mbarrier wait is bounded: a wait that
// runs out marks the partial as NaN (the combine passes NaN to the output)
// and thread 0 still waits, bounded, for the CTA's copies before the CTA
// exits.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <string.h>

#include <mutex>

#include "kvq_batch_splits.h"
#include "kvq_internal.cuh"
#include "kvq_ptx.cuh"
#include "kvq_tanh.cuh"

// This file is compiled three times.  As it stands it is the dense decode;
// included by kvq_decode_lists.cu with KVQ_DECODE_LISTS set it is the decode
// over block lists (kvq_sparse_decode_attn), whose work items are described at
// DecodeArgs; included by kvq_decode_scores.cu with KVQ_DECODE_SCORES set it
// is the dense decode with capped, biased and windowed scores
// (kvq_decode_attn_scored).
#ifndef KVQ_DECODE_LISTS
#define KVQ_DECODE_LISTS 0
#endif
#ifndef KVQ_DECODE_SCORES
#define KVQ_DECODE_SCORES 0
#endif

namespace kvq {
namespace {

constexpr bool kLists = KVQ_DECODE_LISTS != 0;
constexpr bool kScores = KVQ_DECODE_SCORES != 0;
constexpr int kConsumerWarps = 4;
constexpr int kThreads = kConsumerWarps * 32;  // thread 0 also issues the copies
constexpr int kTC = 64;                      // cells per pipeline stage (a piece index is
                                             // split by shifts: 64 = 2^6)
constexpr int kCellsPerWarp = kTC / kConsumerWarps;
constexpr float kTau = 8.0f;                 // lazy rescale threshold (log2 units)
// A raised reference maximum lies this far below the row's own (log2 units),
// so p runs up to 2^kTau.  Dense: 0.  Block lists: kTau, which keeps the fp16
// lo halves of p (times the V scale, often below 0.05) clear of fp16's
// subnormals (int8 cache, 16 ragged lists of 4096 cells: relative output
// error 3.2e-6 without, below 1e-6 with it) at the price of a rescale
// whenever the maximum rises at all.  Scored decode: as block lists.
constexpr float kBelowMax = kLists || kScores ? kTau : 0.0f;
// int8 and K8V4 fold the V scale into p before the fp16 split: 2^kTau times a
// scale of kScaleMost stays below fp16's 65504.  Cells with a larger one have
// p at most 1 (see softmax).  Looking for them costs the dense decode 0-1 %
// (int8 with head_dim 64, whose tiles are the shortest, 1-6 %: 8 sequences of
// 8192 cells x 8 heads 29.7 -> 31.5 us).
constexpr uint32_t kScaleMost = 0x5800u;   // fp16 bits of 128
// int8 K in q.k.  Dense: as 1152 + code, the 1152 * sum(q) taken off through
// the accumulator's start (no subtraction per element).  The sums then run
// at 1152 times the codes' weight and leave a logit error of up to about
// 1e-5; block lists and scored decode subtract first (4 HSUB2 more per 16 x
// 16 tile) and keep it at the FP16 cache's 1e-6.
constexpr bool kCodesExact = kLists || kScores;
constexpr unsigned kFull = 0xffffffffu;

template <int FMT, int HD, int NT>
struct Cfg {
  static constexpr bool KI8 = FMT != KVQ_F16;            // K as int8 codes + scales
  static constexpr bool V4 = FMT == KVQ_K8V4;            // V as rotated 4-bit codes
  static constexpr int ESZ = FMT == KVQ_F16 ? 2 : 1;
  static constexpr int ROWB = HD * ESZ;                  // K code bytes per cell row
  static constexpr int SWB = ROWB < 128 ? ROWB : 128;    // swizzle span (64 or 128 B)
  static constexpr int NCH = ROWB / SWB;                 // swizzle spans per row
  static constexpr int NG = HD / kGroup;
  static constexpr int VROWB = V4 ? HD / 2 : ROWB;       // V code bytes per cell row
  static constexpr int VSWB = VROWB < 128 ? VROWB : 128; // (32, 64 or 128 B)
  static constexpr int VNCH = VROWB / VSWB;
  static constexpr int VNS = V4 ? HD / kQ4Block : NG;    // V scales per cell row
  static constexpr int TILE_B = kTC * ROWB;              // K codes of a stage
  static constexpr int VTILE_B = kTC * VROWB;            // V codes of a stage
  static constexpr int KSCALE_B = KI8 ? kTC * NG * 2 : 0;
  static constexpr int VSCALE_B = KI8 ? kTC * VNS * 2 : 0;
  static constexpr int SC_STAGE_B = KSCALE_B + VSCALE_B;
  // A stage holds the K and V code tiles (each a whole number of 1 KB
  // swizzle atoms); the scales of all stages live in a region of their
  // own so no stage is padded.
  static constexpr int STAGE_B = TILE_B + VTILE_B;
  // Three stages per CTA (one landing while two are read) and as many
  // 4-warp CTAs per SM as the 227 KB allow keep about 100 KB or more of
  // copies in flight per SM.
  // (the merge at the end reuses the stages for 4 warp slabs of RP x HD
  // fp32, which takes a fourth stage for 32-row int8 HD 64 tiles)
  static constexpr int SLAB_B = kConsumerWarps * NT * 8 * HD * 4;
  // Scored, head_dim 256 of int8 keys: two stages where that is one more CTA an SM
  // (K8V4 with 8 rows: 3; int8 with 16: 2), since warps that are ready, not
  // copies under way, are what they lack (2 x 98000 cells, 2 heads, 32 rows, blocks of 256: int8
  // 118 us with 8 rows a CTA and 3 stages, 146 with 16 and 3, 101 with 16 and 2).
  // FP16 of head_dim 128 with 16 rows: two stages and three CTAs likewise (16 ragged
  // sequences, 12 or 16 rows 125 and 130 us -> 123 and 126, 32 rows of half the heads
  // 130 -> 123; with 4 rows it loses, 99 -> 102).
  static constexpr bool TWO = kScores && (HD == 256 ? (V4 ? NT == 1 : KI8 && NT == 2) : HD == 128 && !KI8 && NT == 2);
  static constexpr int STAGES = TWO ? 2 : (SLAB_B + STAGE_B - 1) / STAGE_B > 3 ? (SLAB_B + STAGE_B - 1) / STAGE_B : 3;
  static constexpr int OFF_V = TILE_B;
  static constexpr int SMEM_SC = STAGES * STAGE_B;  // [STAGES]{K [64][NG], V [64][VNS]} fp16
  // q as fp16 hi / lo rows, padded by 16 bytes so ldmatrix rows hit distinct banks
  static constexpr int QROW = HD * 2 + 16;
  static constexpr int QBYTES_MAX = 2 * NT * 8 * QROW;   // hi and lo, NT*8 padded rows
  static constexpr int SMEM_Q = SMEM_SC + STAGES * SC_STAGE_B;
  // int8, dense: per (padded row, 64-dim group, 32-dim half) 1152 * sum of q (hi + lo)
  static constexpr int SMEM_QC = SMEM_Q + (QBYTES_MAX + 15) / 16 * 16;
  static constexpr int QC_BYTES = KI8 && !kCodesExact ? (NT * 8 * NG * 2 * 4 + 15) / 16 * 16 : 0;
  // per-warp row maxima and sums for the merge at the end: [4][RP][2] fp32
  static constexpr int SMEM_WML = SMEM_QC + QC_BYTES;
  static constexpr int SMEM_BAR = SMEM_WML + kConsumerWarps * NT * 8 * 2 * 4;
  // block ids of the split's pieces, staged once so any warp can issue a refill
  static constexpr int ROWS_CAP = 128;
  // (scored: room for a barrier for each warp's slice of each stage)
  static constexpr int SMEM_REL = SMEM_BAR + STAGES * 8 * (kScores ? kConsumerWarps : 1);  // release counters [STAGES]
  static constexpr int SMEM_BLK = SMEM_REL + 16 * 4;            // block ids [ROWS_CAP]
  static constexpr int SMEM = SMEM_BLK + ROWS_CAP * 4 + 1024 /*align*/;
  static constexpr int FIT = (228 * 1024) / (SMEM + 1024);  // 1 KB reserved per CTA
  // 32-row tiles (NT 4) hold 4x the accumulators: at most 3 CTAs (168
  // registers a thread) so they do not spill
  // (K8V4's 16-row tiles, whose smaller stages would fit 4, likewise)
  static constexpr int FIT_R = (NT >= 4 || (V4 && NT >= 2)) ? (FIT < 3 ? FIT : 3) : FIT;
  static constexpr int MIN_CTAS = FIT_R >= 4 ? 4 : (FIT_R >= 3 ? 3 : (FIT_R >= 2 ? 2 : 1));
  static_assert(STAGES * STAGE_B >= SLAB_B, "merge slabs fit in the stages");
  // the SM's 228 KB hold MIN_CTAS of these CTAs (1 KB of each is reserved)
  static_assert(MIN_CTAS * (SMEM + 1024) <= 228 * 1024, "CTAs per SM fit the shared memory");
};

// One 2D tensor map per SWB-byte span of a cell row: [rows][SWB], row
// stride = the row's bytes.  A piece of pc cells lands as [span][cell][SWB].
struct TmaMaps {
  CUtensorMap k[4];
  CUtensorMap v[4];
};

// int8 -> fp16, exactly: with u = c ^ 0x80 (= c + 128 as an unsigned byte),
// the fp16 bit pattern 0x6400 | u is 1024 + u, and (1024 + u) - 1152 = c.
constexpr uint32_t kMagic = 0x64646464u;
constexpr uint32_t kBias = 0x64806480u;  // fp16 1152 in both halves

// Swizzled shared-memory byte offset of logical byte `b` of cell `c` (0..63)
// in a K or V tile laid out [span][cell][SWB]: every TMA box (one piece of
// cells, one span) is placed at its [span][first cell] slot, so the layout
// and the swizzle (XOR of the 16-byte chunk with the line index mod 8 or 4)
// do not depend on the block size.
__device__ __forceinline__ uint32_t swz_off(int c, int b, int sw) {
  const uint32_t off = ((uint32_t)(b / sw) * kTC + (uint32_t)c) * sw + (uint32_t)(b % sw);
  // 128-byte swizzle: chunk bits [4:6] ^= address bits [7:9]; 64-byte:
  // [4:5] ^= [7:8]; 32-byte: [4] ^= [7]
  return off ^ (((off >> 7) & (uint32_t)(sw / 16 - 1)) << 4);
}

template <int FMT, int HD>
__device__ __forceinline__ uint32_t tile_off(int c, int b) {
  return swz_off(c, b, Cfg<FMT, HD, 1>::SWB);
}

// r / G for a query row index r (r < 32 <= 2^32 / G): a multiply by the
// host's ceil(2^32 / G) instead of a division by a run-time value, which
// sat on the path to each CTA's first copy (8 q loads a thread, each with
// a row index to divide)
__device__ __forceinline__ int div_g(const DecodeArgs& a, int r) {
  return (int)(((unsigned long long)(unsigned)r * a.g_magic) >> 32);
}

__device__ __forceinline__ int clamp_len_mma(int L, const DecodeArgs& a) {
  const long long cap_table = (long long)a.max_blocks << a.pool.bs_log2;
  const long long cap_plan = (long long)a.nsplit * a.split_cells;
  const long long cap = cap_table < cap_plan ? cap_table : cap_plan;
  return L < 0 ? 0 : (int)((long long)L < cap ? L : cap);
}

// First and last cell of a sequence's splits.  Scored decode: the first is the
// tile that holds the first cell any of its query tokens sees (the window's
// first token's).
struct Span {
  int base, end;
};

// first cell that query token w of sequence b sees
__device__ __forceinline__ int first_seen(const DecodeArgs& a, int b, int L, int w) {
  int lo = a.first != nullptr ? max(__ldg(a.first + b), 0) : 0;
  if (a.window > 0) lo = (int)max((long long)lo, (long long)L - a.W + w - a.window + 1);
  return lo;
}

__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b, int L_raw) {
  if (!kScores || a.whole) return {0, clamp_len_mma(L_raw, a)};
  const long long cap = (long long)a.max_blocks << a.pool.bs_log2;
  const int L = L_raw < 0 ? 0 : (int)min((long long)L_raw, cap);
  const int base = min(first_seen(a, b, L, 0), L) & ~(kTC - 1);
  return {base, (int)min((long long)L, base + (long long)a.nsplit * a.split_cells)};
}

// The cell count the query tokens' positions go by (span_of's end may be cut
// short by the plan, this is not).
__device__ __forceinline__ int context_of(const DecodeArgs& a, int L_raw) {
  if (!kScores || a.whole) return clamp_len_mma(L_raw, a);
  const long long cap = (long long)a.max_blocks << a.pool.bs_log2;
  return L_raw < 0 ? 0 : (int)min((long long)L_raw, cap);
}

// Block id of cell c (-1 past the end).  Loaded a tile ahead of its use and
// only tested when used, so the load latency stays hidden.
__device__ __forceinline__ int block_of(const DecodeArgs& a, const int32_t* bt, int c, int c_end) {
  return c < c_end ? __ldg(bt + (c >> a.pool.bs_log2)) : -1;
}

// Work item of CTA c.  The grid is one CTA per possible (sequence, KV head,
// split); the items that hold cells are numbered so that every full-length
// split comes first (in sequence, split, KV head order) and the last,
// shorter split of each sequence after them.  CTAs are dispatched roughly in
// index order, so the short splits fill the tail of the launch instead of
// full-length splits starting last.  Every warp computes this itself, a
// warp-wide scan over 32 sequences at a time.  Returns false past the end.
__device__ __forceinline__ bool item_of(const DecodeArgs& a, int c, int& b, int& kvh, int& split) {
  const int lane = threadIdx.x & 31;
  const int S = a.split_cells, nkv = a.n_kv;
  for (int pass = 0; pass < 2; ++pass) {   // 0: full splits, 1: last partial splits
    for (int b0 = 0; b0 < a.n_seq; b0 += 32) {
      const int bb = b0 + lane;
      int n = 0, Lb = 0;
      if (bb < a.n_seq) {
        const Span sp = span_of(a, bb, __ldg(a.ctx_lens + bb));
        Lb = sp.end - sp.base;
        const int qs = (int)fdiv((unsigned)Lb, a.div_split);   // Lb / S (Lb >= 0)
        n = pass == 0 ? qs * nkv : (Lb - qs * S != 0 ? nkv : 0);
      }
      int incl = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += y;
      }
      const int total = __shfl_sync(kFull, incl, 31);
      if (c < total) {
        const unsigned m = __ballot_sync(kFull, bb < a.n_seq && incl > c);
        const int src = __ffs(m) - 1;
        const int k = c - __shfl_sync(kFull, incl - n, src);
        const int Ls = __shfl_sync(kFull, Lb, src);
        b = b0 + src;
        if (pass == 0) {
          split = (int)fdiv((unsigned)k, a.div_nkv);
          kvh = k - split * nkv;
        } else {
          split = (int)fdiv((unsigned)Ls, a.div_split);
          kvh = k;
        }
        return true;
      }
      c -= total;
    }
  }
  return false;
}

// Scored batches: the tiles of sequences lane + 32 i, the split length chosen
// from them, and the item of CTA c (false: past the last): full splits first,
// as above; slot: its number among the splits of its KV head.
struct Batch {
  int tiles[kBatchMaxSeq / 32];
  int split;   // tiles
};

__device__ __forceinline__ int sum_splits(const DecodeArgs& a, const Batch& t, int split, int below) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kBatchMaxSeq / 32; ++i)
    if (32 * i < a.n_seq && lane + 32 * i < below) n += (t.tiles[i] + split - 1) / split;
  return __reduce_add_sync(kFull, n);
}

__device__ __forceinline__ Batch batch_of(const DecodeArgs& a) {
  const int lane = threadIdx.x & 31;
  Batch t;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kBatchMaxSeq / 32; ++i) {
    const int b = lane + 32 * i;
    t.tiles[i] = 0;
    if (b < a.n_seq) {
      const Span sp = span_of(a, b, __ldg(a.ctx_lens + b));
      t.tiles[i] = (sp.end - sp.base + kTC - 1) / kTC;
    }
    n += t.tiles[i];
  }
  t.split = batch_split((long long)__reduce_add_sync(kFull, n), a.batch_items, a.n_seq,
                        [&](int s) { return sum_splits(a, t, s, a.n_seq); });
  return t;
}

__device__ __forceinline__ bool batch_item(const DecodeArgs& a, const Batch& t, int c, int& b, int& kvh, int& split,
                                           int& slot) {
  const int lane = threadIdx.x & 31;
  int k = (int)fdiv((unsigned)c, a.div_nkv);
  kvh = c - k * a.n_kv;
  for (int pass = 0; pass < 2; ++pass) {   // 0: full splits, 1: last partial splits
#pragma unroll
    for (int i = 0; i < kBatchMaxSeq / 32; ++i) {
      if (32 * i >= a.n_seq) break;
      const int full = t.tiles[i] / t.split;
      const int n = pass == 0 ? full : t.tiles[i] - full * t.split != 0;
      int incl = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += y;
      }
      const unsigned m = __ballot_sync(kFull, incl > k);
      if (m != 0) {
        const int src = __ffs(m) - 1;
        const int before = __shfl_sync(kFull, incl - n, src), q = __shfl_sync(kFull, full, src);
        b = 32 * i + src;
        split = pass == 0 ? k - before : q;
        slot = sum_splits(a, t, t.split, b) + split;
        return true;
      }
      k -= __shfl_sync(kFull, incl, 31);
    }
  }
  return false;
}

// ---------------------------------------------------------------------------
// Block lists, the splits of a row tile in one thread-block cluster: the CTAs'
// rows meet through distributed shared memory and the output is written
// here, without partials in global memory and a second kernel.  Called after
// the 4 warps' slabs are in place; leaves when every CTA has read its peers.
// ---------------------------------------------------------------------------
template <int FMT, int HD, int NT>
__device__ __forceinline__ void merge_cluster(const DecodeArgs& a, unsigned char* smem, int list, int r0, int Rc) {
  using C = Cfg<FMT, HD, NT>;
  constexpr int RP = NT * 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* s_slab = reinterpret_cast<float*>(smem);                          // [warp][Rc][HD]
  const float* s_wml = reinterpret_cast<const float*>(smem + C::SMEM_WML);  // [warp][RP][m, l]
  float2* s_fin = reinterpret_cast<float2*>(smem + C::SMEM_Q);             // [Rc] (q is done with)
  // this CTA's rows, in slab 0, and their maximum (NaN: a lost wait) and sum
  if constexpr (C::V4) {
    constexpr int U = HD >= 128 ? 4 : 2, NI = HD / (32 * U);
    for (int r = warp; r < Rc; r += kConsumerWarps) {
      float x[NI][U];
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const float* col = s_slab + r * HD + U * lane + 32 * U * i + e;
          x[i][e] = (col[0] + col[Rc * HD]) + (col[2 * Rc * HD] + col[3 * Rc * HD]);
        }
      wht_warp<U, NI>(x, lane);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < U; ++e) s_slab[r * HD + U * lane + 32 * U * i + e] = x[i][e] * (1.0f / HD);
    }
  } else {
    float4* s4 = reinterpret_cast<float4*>(s_slab);
    const int n4 = Rc * HD / 4;
    for (int i4 = threadIdx.x; i4 < n4; i4 += kThreads) {
      const float4 v0 = s4[i4], v1 = s4[n4 + i4], v2 = s4[2 * n4 + i4], v3 = s4[3 * n4 + i4];
      s4[i4] = make_float4((v0.x + v1.x) + (v2.x + v3.x), (v0.y + v1.y) + (v2.y + v3.y),
                           (v0.z + v1.z) + (v2.z + v3.z), (v0.w + v1.w) + (v2.w + v3.w));
    }
  }
  if (threadIdx.x < Rc) {
    const int r = threadIdx.x;
    float M = s_wml[r * 2];
    bool bad = M != M;
#pragma unroll
    for (int w = 1; w < kConsumerWarps; ++w) {
      const float mw = s_wml[(w * RP + r) * 2];
      bad |= mw != mw;
      M = fmaxf(M, mw);
    }
    float lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kConsumerWarps; ++w)
      lsum = fmaf(s_wml[(w * RP + r) * 2 + 1], fast_exp2(s_wml[(w * RP + r) * 2] - M), lsum);
    s_fin[r] = make_float2(bad ? __int_as_float(0x7fc00000) : M, lsum);
  }
  __syncthreads();
  const uint32_t n_cta = 1u << a.c_log2, rank = blockIdx.x & (n_cta - 1u);
  if (n_cta > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  const uint32_t fin = smem_u32(s_fin), slab = smem_u32(s_slab);
  auto peer_addr = [](uint32_t addr, uint32_t peer) -> uint32_t {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(peer));
    return r;
  };
  // the cluster's threads share the row tile's float4 columns
  for (int i4 = (int)rank * kThreads + (int)threadIdx.x; i4 < Rc * HD / 4; i4 += (int)n_cta * kThreads) {
    const int r = i4 / (HD / 4);
    float M = -INFINITY, lam = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    bool bad = false;
    constexpr int B = 4;   // peers whose loads are in flight together
    for (uint32_t j0 = 0; j0 < n_cta; j0 += B) {
      float2 ml[B];
      float4 v[B];
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const uint32_t j = min(j0 + u, n_cta - 1u);
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                     : "=f"(ml[u].x), "=f"(ml[u].y)
                     : "r"(peer_addr(fin + 8 * r, j)));
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[u].x), "=f"(v[u].y), "=f"(v[u].z), "=f"(v[u].w)
                     : "r"(peer_addr(slab + 16 * i4, j)));
        if (j0 + u >= n_cta) ml[u] = make_float2(-INFINITY, 0.f);
      }
      float top = M;
#pragma unroll
      for (int u = 0; u < B; ++u) {
        // (a NaN sum: a NaN or infinite logit in a live cell)
        bad |= ml[u].x != ml[u].x || ml[u].y != ml[u].y;
        top = fmaxf(top, ml[u].x);
      }
      const float keep = M == -INFINITY ? 0.f : fast_exp2(M - top);
      acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
      lam *= keep;
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const float w = ml[u].y > 0.f ? fast_exp2(ml[u].x - top) : 0.f;
        if (w > 0.f) {
          acc.x = fmaf(w, v[u].x, acc.x);
          acc.y = fmaf(w, v[u].y, acc.y);
          acc.z = fmaf(w, v[u].z, acc.z);
          acc.w = fmaf(w, v[u].w, acc.w);
          lam = fmaf(w, ml[u].y, lam);
        }
      }
      M = top;
    }
    const float inv = lam > 0.f ? 1.f / lam : 0.f;   // (no cell: 0)
    float4 res = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (bad) {
      const float nan = __int_as_float(0x7fc00000);
      res = make_float4(nan, nan, nan, nan);
    }
    reinterpret_cast<float4*>(a.out + ((size_t)list * a.G + r0) * HD)[i4] = res;
  }
  if (n_cta > 1) {   // the peers may still read this CTA's rows
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
// Who fetches a stage of the scored kernel.  With few rows of short heads the
// four warps keep step, and the last to let a stage go refills all of it in
// pieces of up to 64 cells.  Where a warp has more to do for a tile (more than 4
// query rows, or heads of 256) the warps drift apart, and each refills its own
// slice of 16 cells as soon as it has read it, at four times the copies.
// Sixteen ragged sequences, device us, shared stages against own slices:
//   4 rows, head_dim 128, blocks of 64:  q8 76.1, 78.6; f16 99, 107; k8v4 77, 84
//                         blocks of 16:  q8 86.2, 79.9; f16 114, 109; k8v4 87, 85
//                         (one choice for all block sizes; the larger ones decide)
//   8 rows, head_dim 128, blocks of 64:  48.0, 48.0; 55.6, 55.6; 48.7, 50.0
//                         blocks of 16:  51.8, 47.9; 66.5, 57.0; 53.8, 50.3
//   16 rows, head_dim 128, blocks of 64: 143, 141; 134, 130 (126 in two stages); 151, 149
//                         blocks of 16:  154, 140; 158, 133 (127); 161, 149
// Two sequences of 65536 to 131072 cells, head_dim 256, blocks of 64:
//   32 rows:  117, 104; 181, 139; 124, 113       8 rows:  44.7, 41.8; 55, 53; 45.6, 42
//   (blocks of 16: 145, 112; 239, 155; 151, 122           53.7, 43.5; 84, 58; 52, 45)
template <int HD, bool HL>
constexpr bool kWarpSlices = kScores && (HD == 256 || !HL);

// HL (at most 4 query rows, NT = 1): the MMA's 8 columns carry the hi
// parts of q (and of p) in columns 0-3 and the lo parts in columns 4-7, so
// each k-step of q.k and each m-tile of p.v takes one MMA instead of two;
// the hi and lo sums meet by one shuffle (lanes t and t ^ 2): per tile for
// the logits, once per split for the output.  q's fragments stay in
// registers.
template <int FMT, int HD, int NT, bool HL>
__global__ void __launch_bounds__(kThreads, Cfg<FMT, HD, NT>::MIN_CTAS)
    decode_mma(const __grid_constant__ TmaMaps maps, DecodeArgs a) {
  static_assert(!HL || NT == 1, "hi/lo columns need a single 8-column row tile");
  constexpr bool kSlices = kWarpSlices<HD, HL>;
  using C = Cfg<FMT, HD, NT>;
  constexpr int KS = HD / 16;   // k-steps of q.k, and m-tiles of p.v
  constexpr int RP = NT * 8;    // padded rows
  constexpr int MAXP = kTC / 16;
  constexpr float kNegInf = -INFINITY;
  constexpr float kMStart = -1e30f;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t qbase = sbase + C::SMEM_Q;                 // q hi rows, then lo rows
  const uint32_t bar_full = sbase + C::SMEM_BAR;
  int* s_rel = reinterpret_cast<int*>(smem + C::SMEM_REL);
  int* s_blk = reinterpret_cast<int*>(smem + C::SMEM_BLK);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Launched as a programmatic dependent of the previous kernel on the
  // stream: nothing it may have written is read before this wait.
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k[0])) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v[0])) : "memory");
    // One sequence: while the previous kernel finishes, the first two tiles
    // of this CTA's split are brought into L2.  Only a hint: the block
    // ids read here may still change before the wait below (the copies
    // read them again after the wait), and a prefetch of the wrong rows
    // costs bandwidth, nothing else.
    if (a.n_seq == 1 && a.n_rt == 1 && !kLists && (!kScores || a.whole)) {
      const int split0 = (int)fdiv(blockIdx.x, a.div_nkv), kvh0 = (int)blockIdx.x - split0 * a.n_kv;
      const int c0 = split0 * a.split_cells;
      const int pcl = a.pool.bs_log2 < 6 ? a.pool.bs_log2 : 6;
      const int cap = clamp_len_mma(INT_MAX, a);   // cells the table row can address
      if (c0 < cap) {
        constexpr int kPrefetchTiles = 2;
        for (int p = 0; p < kPrefetchTiles * (kTC >> pcl) && (p << pcl) < a.split_cells && c0 + (p << pcl) < cap;
             ++p) {
          // read at L2 (no L1 line: the reads after the wait must not
          // find a copy taken before the previous kernel's writes)
          const int blk = __ldcg(a.block_table + ((c0 + (p << pcl)) >> a.pool.bs_log2));
          if (blk < 0 || blk >= a.pool.n_blocks) continue;
          const size_t row =
              ((size_t)blk * a.pool.n_kv + kvh0) * (1u << a.pool.bs_log2) + ((c0 + (p << pcl)) & ((1 << a.pool.bs_log2) - 1));
          const uint32_t n = 1u << pcl;
          prefetch_l2(static_cast<const char*>(a.pool.k) + row * C::ROWB, n * C::ROWB);
          prefetch_l2(static_cast<const char*>(a.pool.v) + row * C::VROWB, n * C::VROWB);
          if constexpr (C::KI8) {
            prefetch_l2(a.pool.ks + row * C::NG, n * C::NG * 2);
            prefetch_l2(a.pool.vs + row * C::VNS, n * C::VNS * 2);
          }
        }
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // One sequence: CTA c is split c / n_kv of KV head c % n_kv whatever the
  // context length (the item order below reduces to that), so the block
  // ids and the first copies need not wait for the length, which is only
  // read after them; a split that turns out to lie past the context marks
  // its slots empty.  A batch: CTAs past the last item (splits beyond a
  // sequence's context) have nothing to do; the combine kernel reads only
  // the slots of live splits.
  // Row tiles: a work item's R query rows are cut into tiles of a.RT rows
  // (a verify window wider than one CTA's accumulators), one CTA each; the
  // CTAs of an item are neighbours in the grid, so all but the first find
  // the item's K/V tiles in L2.
  // (block lists in clusters: the CTAs of a cluster are the splits of one row
  // tile)
  const bool clustered = kLists && a.c_log2 >= 0;
  const int tile_id = clustered ? (int)(blockIdx.x >> a.c_log2) : (int)blockIdx.x;
  const int item = (int)fdiv((unsigned)tile_id, a.div_nrt);
  const int r0 = (tile_id - item * a.n_rt) * a.RT;          // first query row of this CTA
  const int Rc = min(a.RT, a.R - r0);                         // and its row count
  int b, kvh, split;
  int L_raw = 0;
  int slot = 0, split_cells = a.split_cells;   // scored batches: chosen below
  // (lists too: their block ids are copied ahead of the length, -1 past the end)
  const bool single = kLists || a.n_seq == 1;
  if (single && !kLists) {
    b = 0;
    split = (int)fdiv((unsigned)item, a.div_nkv);
    kvh = item - split * a.n_kv;
    L_raw = __ldg(a.ctx_lens);
  } else if (kLists) {
    // block lists: split-major, no search (the lists are about equally long)
    split = clustered ? (int)(blockIdx.x & ((1u << a.c_log2) - 1u)) : (int)fdiv((unsigned)item, a.div_nseq);
    b = clustered ? item : item - split * a.n_seq;
    kvh = 0;
    L_raw = __ldg(a.ctx_lens + b);
  } else if (kScores && a.batch_items > 0) {
    const Batch t = batch_of(a);
    split_cells = t.split * kTC;
    if (blockIdx.x == 0) {   // where each sequence's splits begin, for the combine
      for (int s = threadIdx.x >> 5; s <= a.n_seq; s += kConsumerWarps) {
        const int first = sum_splits(a, t, t.split, s);
        if ((threadIdx.x & 31) == 0) a.ws_base[s] = first;
      }
    }
    if (!batch_item(a, t, item, b, kvh, split, slot)) return;
    L_raw = __ldg(a.ctx_lens + b);
  } else {
    if (!item_of(a, item, b, kvh, split)) return;
    L_raw = __ldg(a.ctx_lens + b);
  }
  // the KV head's place in the pool
  const int pool_h = kLists ? b - (int)fdiv((unsigned)b, a.div_heads) * a.pool.n_kv : kvh;
  const Span span = kScores && !a.whole ? span_of(a, b, L_raw) : Span{0, 0};
  const int c_begin = span.base + split * split_cells;
  // until the length is known (one sequence), copies stay inside the split
  // and the block table
  int c_end = min(kScores && !a.whole ? span.end : clamp_len_mma(single ? INT_MAX : L_raw, a),
                  c_begin + split_cells);
  int n_tiles = (c_end - c_begin + kTC - 1) / kTC;
  if ((kLists || kScores) && n_tiles < 0) n_tiles = 0;   // (an empty split of a cluster, or past a window)
  const int n_first = n_tiles < C::STAGES ? n_tiles : C::STAGES;   // tiles of the first wave
  const int pc_log2 = a.pool.bs_log2 < 6 ? a.pool.bs_log2 : 6;  // cells per TMA piece
  const int n_pieces = kTC >> pc_log2;
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;
  const bool producer = threadIdx.x == 0;
  // Dense: the cache is read once per call, so its lines leave L2 first.  (Lists
  // keep the hint, although the tokens of a verify window may share blocks.)
  const uint64_t pol = l2_evict_first_policy();
  // Let the combine grid be scheduled as soon as SMs free up; it still waits
  // (griddepcontrol.wait) for this whole grid to finish before reading.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Copies of a stage are issued by whichever warp releases the stage last
  // (a shared-memory counter per stage), so no warp ever blocks waiting for
  // the others.  The block id of every piece of the split is staged in
  // shared memory once (when it fits), so an issuing warp needs no global
  // load on that path.
  const int n_entries = n_tiles * n_pieces;
  const bool blk_in_smem = n_entries <= C::ROWS_CAP;
  // Scored, with a distance bias: the newest tiles first, whose scores set the
  // maximum (the other way round every tile would raise it).  A split whose length
  // is not known when its first copies go out starts at its beginning.
  const bool newest_first = kScores && a.slopes != nullptr && (!single || !a.whole);
  auto tile_of = [&](int it) -> int { return newest_first ? n_tiles - 1 - it : it; };
  auto piece_blk = [&](int it, int p, bool from_smem) -> int {
    return from_smem ? s_blk[it * n_pieces + p]
                     : block_of(a, bt, c_begin + it * kTC + (p << pc_log2), c_end);
  };
  // block ids of the pieces of tile it
  auto tile_blks = [&](int it, bool from_smem, int (&blk)[MAXP]) {
#pragma unroll
    for (int p = 0; p < MAXP; ++p) blk[p] = p < n_pieces ? piece_blk(it, p, from_smem) : -1;
  };
  auto issue = [&](int it, const int (&blks)[MAXP]) {
    const int s = it % C::STAGES;
    const int pc = 1 << pc_log2;
    const int bsz = 1 << a.pool.bs_log2;
    const int c0 = c_begin + it * kTC;
    int rows[MAXP];
    uint32_t bytes = 0;
#pragma unroll
    for (int p = 0; p < MAXP; ++p) {
      const int blk = blks[p];
      const int c = c0 + (p << pc_log2);
      rows[p] = (p < n_pieces && blk >= 0 && blk < a.pool.n_blocks)
                    ? (blk * a.pool.n_kv + pool_h) * bsz + (c & (bsz - 1))
                    : -1;
      if (rows[p] >= 0) bytes += (uint32_t)pc * (C::ROWB + C::VROWB + (C::KI8 ? (C::NG + C::VNS) * 2 : 0));
    }
    const uint32_t full = bar_full + 8 * s;
    mbar_expect_tx(full, bytes + a.extra_tx);
    const uint32_t st = sbase + s * C::STAGE_B;
    for (int p = 0; p < n_pieces; ++p) {
      const int row = rows[p];
      if (row < 0) continue;
#pragma unroll
      for (int sp = 0; sp < C::NCH; ++sp) {
        const uint32_t so = (uint32_t)(sp * kTC + (p << pc_log2)) * C::SWB;
        tma_load_2d_hint(st + so, &maps.k[sp], 0, row, full, pol);
      }
#pragma unroll
      for (int sp = 0; sp < C::VNCH; ++sp) {
        const uint32_t so = (uint32_t)(sp * kTC + (p << pc_log2)) * C::VSWB;
        tma_load_2d_hint(st + C::OFF_V + so, &maps.v[sp], 0, row, full, pol);
      }
      if constexpr (C::KI8) {
        const uint32_t sbk = (uint32_t)pc * C::NG * 2, sbv = (uint32_t)pc * C::VNS * 2;
        const uint32_t sc = sbase + C::SMEM_SC + (uint32_t)s * C::SC_STAGE_B;
        bulk_load_hint(sc + (uint32_t)p * sbk, a.pool.ks + (size_t)row * C::NG, sbk, full, pol);
        bulk_load_hint(sc + C::KSCALE_B + (uint32_t)p * sbv, a.pool.vs + (size_t)row * C::VNS, sbv, full, pol);
      }
    }
  };

  // Scored: the same by a whole warp, a copy a lane (a stage of blocks of 16 cells
  // is up to 32 copies).
  auto issue_warp = [&](int it, bool from_smem) {
    constexpr int NC = C::NCH + C::VNCH + (C::KI8 ? 2 : 0);   // copies of a piece
    static_assert(!kScores || MAXP * NC <= 32, "a copy a lane");
    const int s = it % C::STAGES;
    const int pc = 1 << pc_log2, bsz = 1 << a.pool.bs_log2;
    const int p = lane / NC, c = lane - p * NC;
    int row = -1;
    uint32_t bytes = 0;
    if (p < n_pieces) {
      const int blk = piece_blk(tile_of(it), p, from_smem), cell = c_begin + tile_of(it) * kTC + (p << pc_log2);
      if (blk >= 0 && blk < a.pool.n_blocks) {
        row = (blk * a.pool.n_kv + pool_h) * bsz + (cell & (bsz - 1));
        bytes = (uint32_t)pc * (c < C::NCH ? C::SWB : c < C::NCH + C::VNCH ? C::VSWB
                                                    : c == NC - 2          ? C::NG * 2
                                                                           : C::VNS * 2);
      }
    }
    const uint32_t full = bar_full + 8 * s, total = __reduce_add_sync(kFull, bytes);
    if (lane == 0) mbar_expect_tx(full, total + a.extra_tx);
    __syncwarp();
    if (row >= 0) {
      const uint32_t st = sbase + s * C::STAGE_B;
      if (c < C::NCH) {
        tma_load_2d_hint(st + (uint32_t)(c * kTC + (p << pc_log2)) * C::SWB, &maps.k[c], 0, row, full, pol);
      } else if (c < C::NCH + C::VNCH) {
        const int sp = c - C::NCH;
        tma_load_2d_hint(st + C::OFF_V + (uint32_t)(sp * kTC + (p << pc_log2)) * C::VSWB, &maps.v[sp], 0, row, full, pol);
      } else if constexpr (C::KI8) {
        const uint32_t sc = sbase + C::SMEM_SC + (uint32_t)s * C::SC_STAGE_B;
        if (c == NC - 2) bulk_load_hint(sc + (uint32_t)p * bytes, a.pool.ks + (size_t)row * C::NG, bytes, full, pol);
        else bulk_load_hint(sc + C::KSCALE_B + (uint32_t)p * bytes, a.pool.vs + (size_t)row * C::VNS, bytes, full, pol);
      }
    }
    __syncwarp();
  };

  // kSlices: each warp fetches its own slice of 16 cells of every stage, a copy a
  // lane, behind a barrier of its own.
  const uint32_t bar_own = kSlices ? bar_full + 8 * C::STAGES * warp : bar_full;
  auto issue_slice = [&](int it, bool from_smem) {
    constexpr int NC = C::NCH + C::VNCH + (C::KI8 ? 2 : 0);   // copies of a slice
    const int s = it % C::STAGES, t = tile_of(it);
    const int bsz = 1 << a.pool.bs_log2, at = warp * kCellsPerWarp;   // the slice in its tile
    const int cell = c_begin + t * kTC + at;
    // (the staged table has an entry a piece of up to 64 cells)
    const int blk = from_smem ? (cell < c_end ? s_blk[t * n_pieces + (at >> pc_log2)] : -1) : block_of(a, bt, cell, c_end);
    const bool there = blk >= 0 && blk < a.pool.n_blocks;
    const uint32_t full = bar_own + 8 * s;
    if (lane == 0)
      mbar_expect_tx(full, (there ? kCellsPerWarp * (C::ROWB + C::VROWB + (C::KI8 ? (C::NG + C::VNS) * 2 : 0)) : 0) + a.extra_tx);
    __syncwarp();
    if (there && lane < NC) {
      const int row = (blk * a.pool.n_kv + pool_h) * bsz + (cell & (bsz - 1)), c = lane;
      const uint32_t st = sbase + s * C::STAGE_B;
      if (c < C::NCH) {
        tma_load_2d_hint(st + (uint32_t)(c * kTC + at) * C::SWB, &maps.k[c], 0, row, full, pol);
      } else if (c < C::NCH + C::VNCH) {
        const int sp = c - C::NCH;
        tma_load_2d_hint(st + C::OFF_V + (uint32_t)(sp * kTC + at) * C::VSWB, &maps.v[sp], 0, row, full, pol);
      } else if constexpr (C::KI8) {
        constexpr uint32_t KB = kCellsPerWarp * C::NG * 2, VB = kCellsPerWarp * C::VNS * 2;
        const uint32_t sc = sbase + C::SMEM_SC + (uint32_t)s * C::SC_STAGE_B;
        if (c == NC - 2) bulk_load_hint(sc + (uint32_t)warp * KB, a.pool.ks + (size_t)row * C::NG, KB, full, pol);
        else bulk_load_hint(sc + C::KSCALE_B + (uint32_t)warp * VB, a.pool.vs + (size_t)row * C::VNS, VB, full, pol);
      }
    }
    __syncwarp();
  };

  // Prologue.  Every small load (q, the split's block ids) is issued first,
  // into registers; only then does thread 0 start the first stages' bulk
  // copies.  Issued the other way round, these few latency-critical loads
  // would queue behind tens of megabytes of copies from all CTAs.
  //
  // q * sm_scale * log2(e) goes to shared memory as fp16 hi + lo, rows
  // [RP][HD] in k order: FP16 uses the natural dim order; int8 permutes each
  // 16-wide k-step ks so that k = 2t + e -> dim 16 ks + 4 t + e and
  // k = 2t + 8 + e -> that + 2 (t = k-pair lane): a lane's ldmatrix word
  // holds the 4 code bytes of dims 16 ks + 4t .. + 3.
  constexpr int QPT = (RP * HD + kThreads - 1) / kThreads;  // q values per thread
  constexpr int BPT = (C::ROWS_CAP + kThreads - 1) / kThreads;
  float qv[QPT];
#pragma unroll
  for (int u = 0; u < QPT; ++u) {
    const int i = threadIdx.x + u * kThreads;
    qv[u] = 0.f;
    if (i < RP * HD) {
      const int r = i / HD, k = i - r * HD;
      int dim = k;
      if constexpr (C::KI8) {
        const int ks = k >> 4, kq = k & 15;
        const int tt = (kq & 7) >> 1, e = kq & 1, hi8 = kq >> 3;
        dim = 16 * ks + 4 * tt + 2 * hi8 + e;
      }
      if (r < Rc) {
        const int w = div_g(a, r0 + r), gg = r0 + r - w * a.G;
        qv[u] = __ldg(a.q + (((size_t)b * a.W + w) * a.n_q + (size_t)kvh * a.G + gg) * HD + dim);
      }
    }
  }
  int bv[BPT];
#pragma unroll
  for (int u = 0; u < BPT; ++u) {
    const int i = threadIdx.x + u * kThreads;
    bv[u] = (blk_in_smem && i < n_entries)
                ? block_of(a, bt, c_begin + (i >> (6 - pc_log2)) * kTC + ((i & (n_pieces - 1)) << pc_log2), c_end)
                : -1;
  }
  bool lost = false;
  if constexpr (kSlices) {
    if (lane == 0) {
      for (int s = 0; s < C::STAGES; ++s) mbar_init(bar_own + 8 * s, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    if (n_first > 0) issue_slice(0, false);
  } else if constexpr (kScores) {
    if (warp == 0) {
      if (lane == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
          mbar_init(bar_full + 8 * s, 1);
          s_rel[s] = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      }
      __syncwarp();
      if (n_first > 0) issue_warp(0, false);
    }
  } else if (producer) {
    // the block ids of every first-wave piece are loaded together, before
    // the first copy is issued
    int fb[C::STAGES][MAXP];
#pragma unroll
    for (int it = 0; it < C::STAGES; ++it) tile_blks(it, false, fb[it]);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      s_rel[s] = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // the first tile now; the rest of the first wave after the barrier
    // below, so that on every SM each CTA's first tile is queued for the
    // copy engine ahead of the other tiles of the wave
    if (n_first > 0) issue(0, fb[0]);
  }
  {
    unsigned char* qs = smem + C::SMEM_Q;
#pragma unroll
    for (int u = 0; u < QPT; ++u) {
      const int i = threadIdx.x + u * kThreads;
      if (i < RP * HD && (!HL || i / HD < 4)) {
        const int r = i / HD, k = i - r * HD;
        const float x = qv[u] * a.qscale;
        const __half h = __float2half_rn(x);
        const __half lo = __float2half_rn(x - __half2float(h));
        *reinterpret_cast<__half*>(qs + r * C::QROW + k * 2) = h;
        *reinterpret_cast<__half*>(qs + (HL ? 4 + r : RP + r) * C::QROW + k * 2) = lo;
        if constexpr (C::KI8 && !kCodesExact) {
          // The 32 lanes of a warp hold 32 consecutive k of one row and one
          // 64-dim group (RP * HD is a multiple of 128): their sum of q,
          // times 1152, fills the (row, group, half) slot of the int8 bias.
          float v = __half2float(h) + __half2float(lo);
#pragma unroll
          for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
          if (lane == 0)
            reinterpret_cast<float*>(smem + C::SMEM_QC)[(r * C::NG + k / 64) * 2 + ((k >> 5) & 1)] =
                1152.0f * v;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < BPT; ++u) {
      const int i = threadIdx.x + u * kThreads;
      if (blk_in_smem && i < n_entries) s_blk[i] = bv[u];
    }
  }
  __syncthreads();
  const int L = context_of(a, L_raw);
  if (single) {
    c_end = min(kScores && !a.whole ? span.end : L, c_begin + split_cells);
    n_tiles = c_end > c_begin ? (c_end - c_begin + kTC - 1) / kTC : 0;
    // (a cluster's empty splits go through the merge with nothing to add)
    if (n_tiles == 0 && !clustered) {
      // a split past the context: its slots tell the combine "no cells"
      if ((kSlices ? lane == 0 : producer) && n_first > 0) (void)mbar_wait(bar_own, 0, a.wait_limit);
      const size_t slot0 = (((size_t)b * a.n_kv + kvh) * a.nsplit + split) * a.R;
      if (threadIdx.x < a.R)
        *reinterpret_cast<float2*>(a.ws_ml + (slot0 + threadIdx.x) * 2) = make_float2(-INFINITY, 0.f);
      return;
    }
  }
  if constexpr (kSlices) {
    for (int it = 1; it < n_first; ++it) issue_slice(it, blk_in_smem);
  } else if (kScores && warp == 0) {
    for (int it = 1; it < n_first; ++it) issue_warp(it, blk_in_smem);
  }
  if (!kScores && producer) {
    for (int it = 1; it < n_first; ++it) {
      int nb[MAXP];
      tile_blks(it, blk_in_smem, nb);
      issue(it, nb);
    }
  }

  // ---------------- consumer setup ----------------
  const int g = lane >> 2, t = lane & 3;

  // Dense: int8 K enters the MMA as fp16 (1152 + code) (no subtraction per
  // element); the 1152 * sum(q) of each (row, 64-dim group) is taken off
  // once, as the starting value of that group's hi accumulator.
  float qcorr[C::KI8 ? C::NG : 1][NT][2];
  if constexpr (C::KI8 && !kCodesExact) {
    const float* s_qc = reinterpret_cast<const float*>(smem + C::SMEM_QC);
#pragma unroll
    for (int gq = 0; gq < C::NG; ++gq)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int i = ((nt * 8 + 2 * t + j) * C::NG + gq) * 2;
          // (HL: the lo columns 4-7 start at 0; the hi ones carry the whole
          // correction, the two meet in the logits)
          qcorr[gq][nt][j] = (HL && t >= 2) ? 0.f : -(s_qc[i] + s_qc[i + 1]);
        }
  }

  // ldmatrix lane addressing of q: matrix lane>>3 = {hi k0-7, hi k8-15, lo
  // k0-7, lo k8-15}, row lane&7.
  const uint32_t q_lane = qbase + (uint32_t)((lane >> 4) * RP + (lane & 7)) * C::QROW +
                          (uint32_t)((lane >> 3) & 1) * 16;
  // HL: the B fragments of every k-step (rows 0-3 hi, 4-7 lo), kept in
  // registers; one ldmatrix x4 covers two k-steps
  uint32_t qreg[HL ? KS : 1][2];
  if constexpr (HL) {
    const uint32_t ql = qbase + (uint32_t)(lane & 7) * C::QROW + (uint32_t)(lane >> 3) * 16;
#pragma unroll
    for (int ks = 0; ks < KS; ks += 2) {
      uint32_t r4[4];
      ldsm_x4(r4, ql + ks * 32);
      qreg[ks][0] = r4[0];
      qreg[ks][1] = r4[1];
      qreg[ks + 1][0] = r4[2];
      qreg[ks + 1][1] = r4[3];
    }
  }

  // Last visible cell of each of this thread's rows (the verify window's
  // causal limit), or -1 for padding rows.
  // the query row of this thread's column j of row tile nt (HL: lanes t
  // and t ^ 2 hold the same rows, hi and lo halves)
  auto row_of = [&](int nt, int j) -> int { return HL ? 2 * (t & 1) + j : nt * 8 + 2 * t + j; };
  int row_last[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = row_of(nt, j);
      row_last[nt][j] = r < Rc ? L - a.W + div_g(a, r0 + r) : -1;
    }

  int row_last_min = INT_MAX;  // smallest causal limit among this thread's real rows
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (row_of(nt, j) < Rc) row_last_min = min(row_last_min, row_last[nt][j]);

  // Scored: the first cell each row sees, its slope (log2 domain), and its
  // position before the context's end
  int row_lo[kScores ? NT : 1][2], row_lo_max = 0, lo_all = 0;
  float row_slope[kScores ? NT : 1][2], row_back[kScores ? NT : 1][2];
  if constexpr (kScores) {
    lo_all = first_seen(a, b, L, 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = row_of(nt, j), w = div_g(a, r0 + r);
        row_lo[nt][j] = r < Rc ? first_seen(a, b, L, w) : 0;
        row_lo_max = max(row_lo_max, row_lo[nt][j]);
        row_back[nt][j] = (float)(a.W - w);
        row_slope[nt][j] = r < Rc && a.slopes != nullptr
                               ? 1.4426950408889634f * __ldg(a.slopes + kvh * a.G + (r0 + r - w * a.G))
                               : 0.f;
      }
  }

  float m[NT][2], l[NT][2];
  float o[KS][NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    // a finite start, so p needs no "no maximum yet" test: the first tile
    // with a visible cell always raises it
    m[nt][0] = m[nt][1] = kMStart;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
  }

  const int cl = warp * kCellsPerWarp;  // first cell of this warp's slice in a stage
  auto slice_blk = [&](int it) -> int {
    if (it >= n_tiles) return -1;
    const int t = tile_of(it);
    if (blk_in_smem) return c_begin + t * kTC + cl < c_end ? s_blk[t * n_pieces + (cl >> pc_log2)] : -1;
    return block_of(a, bt, c_begin + t * kTC + cl, c_end);
  };
  auto slice_nvalid = [&](int it, int blk) -> int {
    return (blk >= 0 && blk < a.pool.n_blocks) ? min(kCellsPerWarp, c_end - (c_begin + tile_of(it) * kTC + cl)) : 0;
  };

  // Swizzled shared-memory addresses.  With a 128-byte swizzle the XOR term
  // of every address this thread reads splits into a per-thread constant and
  // a compile-time part, so a few base registers replace the full
  // computation per load (the spans of a row are whole 64-cell x 128-byte
  // blocks, reached by immediate offsets).
  //
  // ldmatrix x4 lane addressing: matrix mi = lane >> 3 reads row rr = lane & 7.
  // kx: matrices (cells +0, chunk 2k), (cells +8, chunk 2k), (cells +0,
  // chunk 2k+1), (cells +8, chunk 2k+1) of the k-th 32-byte step of a row --
  // K for q.k in both formats and, as byte pairs, int8 V for p.v.  vx (FP16
  // V^T): (cells +0, chunk 2k), (+0, 2k+1), (+8, 2k), (+8, 2k+1).
  constexpr uint32_t kSpanB = kTC * 128;
  uint32_t kx[4], vx[4];
  {
    const int mi = lane >> 3, rr = lane & 7;
    const uint32_t ck = (uint32_t)(cl + ((mi & 1) << 3) + rr), cv = (uint32_t)(cl + ((mi >> 1) << 3) + rr);
    if constexpr (C::SWB == 128) {
      const uint32_t xk = ((uint32_t)(mi >> 1) << 4) ^ ((uint32_t)rr << 4);
      const uint32_t xv = ((uint32_t)(mi & 1) << 4) ^ ((uint32_t)rr << 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        kx[k] = ck * 128 + (xk ^ (32u * k));
        vx[k] = C::OFF_V + cv * 128 + (xv ^ (32u * k));
      }
    } else {  // 64-byte rows (int8, HD 64): two 32-byte steps
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        kx[k] = tile_off<FMT, HD>((int)ck, (32 * k + 16 * (mi >> 1)) & (C::ROWB - 1));
        vx[k] = 0;
      }
    }
  }
  // K8V4 V: the same matrix order over 16-byte chunks of the nibble rows
  // (chunk = one 32-dim block), in the V tile's own swizzle span.
  uint32_t vq[C::V4 ? C::VROWB / 32 : 1];
  if constexpr (C::V4) {
    const int mi = lane >> 3, rr = lane & 7;
    const int ck = cl + ((mi & 1) << 3) + rr;
#pragma unroll
    for (int k = 0; k < C::VROWB / 32; ++k) vq[k] = C::OFF_V + swz_off(ck, 32 * k + 16 * (mi >> 1), C::VSWB);
  }
  // shared-memory offset of the k-th 32-byte step of the kx row set
  auto kstep = [&](int k) -> uint32_t {
    if constexpr (C::SWB == 128) return kx[k & 3] + (uint32_t)(k >> 2) * kSpanB;
    else return kx[k & 1];
  };

  // q . k of one stage for this warp's 16 cells -> z (log2-domain logits)
  auto qk = [&](int s, float (&z)[NT][4]) {
    const uint32_t st = sbase + s * C::STAGE_B;
  // ---------------- S^T = K . Q^T (four independent accumulators) ----------------
  if constexpr (FMT == KVQ_F16 && HL) {
    float acc[2][4];  // alternate k-steps, two independent chains
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t af[4];
      ldsm_x4(af, st + kx[ks & 3] + (uint32_t)(ks >> 2) * kSpanB);
      if (ks < 2) mma16816_zc(acc[ks & 1], af, qreg[ks][0], qreg[ks][1]);
      else mma16816(acc[ks & 1], af, qreg[ks][0], qreg[ks][1]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float v = acc[0][k] + acc[1][k];
      z[0][k] = v + __shfl_xor_sync(kFull, v, 2);  // hi columns + lo columns
    }
  } else if constexpr (FMT == KVQ_F16) {
    float acc[4][NT][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t af[4];
      ldsm_x4(af, st + kx[ks & 3] + (uint32_t)(ks >> 2) * kSpanB);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t qf[4];
        ldsm_x4(qf, q_lane + (uint32_t)(nt * 8) * C::QROW + ks * 32);
        if (ks < 2) {
          mma16816_zc(acc[(ks & 1) * 2 + 0][nt], af, qf[0], qf[1]);
          mma16816_zc(acc[(ks & 1) * 2 + 1][nt], af, qf[2], qf[3]);
        } else {
          mma16816(acc[(ks & 1) * 2 + 0][nt], af, qf[0], qf[1]);
          mma16816(acc[(ks & 1) * 2 + 1][nt], af, qf[2], qf[3]);
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        z[nt][k] = (acc[0][nt][k] + acc[2][nt][k]) + (acc[1][nt][k] + acc[3][nt][k]);
  } else {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) z[nt][0] = z[nt][1] = z[nt][2] = z[nt][3] = 0.f;
    const unsigned short* ksc = reinterpret_cast<const unsigned short*>(smem + C::SMEM_SC + s * C::SC_STAGE_B);
#pragma unroll
    for (int gq = 0; gq < C::NG; ++gq) {
      // words: [k-step kk][cells +0 | +8], each the 4 code bytes of dims
      // 16 (4 gq + kk) + 4t .. + 3 of cell g (or g + 8)
      uint32_t w[4][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[4];
        ldsm_x4(r, st + kstep(2 * gq + h));
        w[2 * h][0] = r[0] ^ 0x80808080u;
        w[2 * h][1] = r[1] ^ 0x80808080u;
        w[2 * h + 1][0] = r[2] ^ 0x80808080u;
        w[2 * h + 1][1] = r[3] ^ 0x80808080u;
      }
      float acc[2][NT][4];  // hi chain (dense: starts at -1152 sum q), lo chain
      if constexpr (!kCodesExact) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[0][nt][0] = acc[0][nt][2] = qcorr[gq][nt][0];
          acc[0][nt][1] = acc[0][nt][3] = qcorr[gq][nt][1];
        }
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        uint32_t af[4];  // fp16 1152 + code (lists: code), exact
        af[0] = prmt(w[kk][0], kMagic, 0x4140u);
        af[2] = prmt(w[kk][0], kMagic, 0x4342u);
        af[1] = prmt(w[kk][1], kMagic, 0x4140u);
        af[3] = prmt(w[kk][1], kMagic, 0x4342u);
        if constexpr (kCodesExact) {
#pragma unroll
          for (int i = 0; i < 4; ++i) af[i] = hsub2(af[i], kBias);
        }
        if constexpr (HL) {
          // one chain: columns 0-3 hi (dense: start at -1152 sum q), 4-7 lo (at 0)
          if (kCodesExact && kk == 0) mma16816_zc(acc[0][0], af, qreg[gq * 4][0], qreg[gq * 4][1]);
          else mma16816(acc[0][0], af, qreg[gq * 4 + kk][0], qreg[gq * 4 + kk][1]);
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t qf[4];
            ldsm_x4(qf, q_lane + (uint32_t)(nt * 8) * C::QROW + (gq * 4 + kk) * 32);
            if (kCodesExact && kk == 0) mma16816_zc(acc[0][nt], af, qf[0], qf[1]);
            else mma16816(acc[0][nt], af, qf[0], qf[1]);
            if (kk == 0) mma16816_zc(acc[1][nt], af, qf[2], qf[3]);
            else mma16816(acc[1][nt], af, qf[2], qf[3]);
          }
        }
      }
      const float s0 = __half2float(__ushort_as_half(ksc[(cl + g) * C::NG + gq]));
      const float s8 = __half2float(__ushort_as_half(ksc[(cl + g + 8) * C::NG + gq]));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (HL) {
          z[nt][0] = fmaf(s0, acc[0][nt][0], z[nt][0]);
          z[nt][1] = fmaf(s0, acc[0][nt][1], z[nt][1]);
          z[nt][2] = fmaf(s8, acc[0][nt][2], z[nt][2]);
          z[nt][3] = fmaf(s8, acc[0][nt][3], z[nt][3]);
        } else {
          z[nt][0] = fmaf(s0, acc[0][nt][0] + acc[1][nt][0], z[nt][0]);
          z[nt][1] = fmaf(s0, acc[0][nt][1] + acc[1][nt][1], z[nt][1]);
          z[nt][2] = fmaf(s8, acc[0][nt][2] + acc[1][nt][2], z[nt][2]);
          z[nt][3] = fmaf(s8, acc[0][nt][3] + acc[1][nt][3], z[nt][3]);
        }
      }
    }
    if constexpr (HL) {
#pragma unroll
      for (int k = 0; k < 4; ++k) z[0][k] += __shfl_xor_sync(kFull, z[0][k], 2);  // hi + lo columns
    }
  }

  };

  // The V scales of this thread's cells g and g + 8, two fp16 a word, read with
  // the slice's K and kept until its p.v.
  constexpr int VSW = C::KI8 ? (C::VNS + 1) / 2 : 1;
  auto load_scales = [&](int s, uint32_t (&vw)[2][VSW]) {
    if constexpr (C::KI8) {
      const unsigned char* vsc = smem + C::SMEM_SC + s * C::SC_STAGE_B + C::KSCALE_B;
#pragma unroll
      for (int ci = 0; ci < 2; ++ci) {
        const unsigned char* src = vsc + (cl + g + 8 * ci) * (C::VNS * 2);
        if constexpr (C::VNS == 1) {
          vw[ci][0] = *reinterpret_cast<const unsigned short*>(src);
        } else if constexpr (VSW == 1) {
          vw[ci][0] = *reinterpret_cast<const uint32_t*>(src);
        } else if constexpr (VSW == 2) {
          const uint2 u = *reinterpret_cast<const uint2*>(src);
          vw[ci][0] = u.x;
          vw[ci][VSW - 1] = u.y;
        } else {
          const uint4 u = *reinterpret_cast<const uint4*>(src);
          vw[ci][0] = u.x;
          vw[ci][VSW > 1 ? 1 : 0] = u.y;
          vw[ci][VSW > 2 ? 2 : 0] = u.z;
          vw[ci][VSW > 3 ? 3 : 0] = u.w;
        }
      }
    }
  };

  // causal / length masks, online softmax -> p (rescales o when the maximum
  // rises).  A lane whose live cells have a V scale above kScaleMost asks for a
  // reference maximum no lower than their logits, so that p (at most 1 then)
  // times the scale is an fp16 number.
  auto softmax = [&](int nvalid, int cw0, const uint32_t (&vw)[2][VSW], float (&z)[NT][4], float (&p)[NT][4]) {
    bool large = false;
    if constexpr (C::KI8) {
      // a half above kScaleMost plus the constant carries into bit 15, and no
      // further
      uint32_t x[2] = {0, 0};
#pragma unroll
      for (int ci = 0; ci < 2; ++ci)
#pragma unroll
        for (int i = 0; i < VSW; ++i) x[ci] |= (vw[ci][i] & 0x7fff7fffu) + (0x7fff7fffu - kScaleMost * 0x10001u);
      if (nvalid < kCellsPerWarp) {   // (the scales of masked cells may be anything)
        if (g >= nvalid) x[0] = 0;
        if (g + 8 >= nvalid) x[1] = 0;
      }
      if (kScores && lo_all > cw0) {
        if (g < lo_all - cw0) x[0] = 0;
        if (g + 8 < lo_all - cw0) x[1] = 0;
      }
      large = ((x[0] | x[1]) & 0x80008000u) != 0;
    }
    const float tau = large ? 0.f : kTau;
    // padding rows never reach the output, so only a short slice or a causal
    // limit inside it needs masks
    const bool need_mask = nvalid < kCellsPerWarp || row_last_min - cw0 < kCellsPerWarp - 1 ||
                           (kScores && row_lo_max > cw0);
    if constexpr (kScores) {
      if (a.cap2 != 0.f) {
        float most = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; k += 2) most = max3f(most, fabsf(z[nt][k]), fabsf(z[nt][k + 1]));
        if (__any_sync(kFull, most > kTanhSmall * a.cap2)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              float s0 = z[nt][k], s1 = z[nt][k + 1];
              cap_small(s0, s1, a.cap2_inv);
              z[nt][k] = cap_any(z[nt][k], s0, a.cap2, a.cap2_inv);
              z[nt][k + 1] = cap_any(z[nt][k + 1], s1, a.cap2, a.cap2_inv);
            }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; k += 2) cap_small(z[nt][k], z[nt][k + 1], a.cap2_inv);
        }
      }
      if (a.slopes != nullptr) {
        const float at = (float)(cw0 + g - L);   // of cell g; a row's position is L - its row_back
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float d = at + row_back[nt][j];   // cell - position: <= 0 where it is seen
            z[nt][j] = fmaf(row_slope[nt][j], d, z[nt][j]);
            z[nt][2 + j] = fmaf(row_slope[nt][j], d + 8.0f, z[nt][2 + j]);
          }
      }
    }
  // ---------------- masks and online softmax ----------------
  // A row's maximum over the slice (8 lanes) is needed only when the
  // reference maximum must rise; that happens only if some lane's own
  // maximum lies above it by more than kTau, so one warp vote decides
  // whether the shuffles run at all (the outcome is the same either way).
  // p is first computed against the current reference maximum, ahead of
  // the vote, so its exponentials need not wait for the branch; the rare
  // tile that raises the maximum computes p again.
  auto probs = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        p[nt][j] = fast_exp2(z[nt][j] - m[nt][j]);
        p[nt][2 + j] = fast_exp2(z[nt][2 + j] - m[nt][j]);
      }
  };
  float lmax[NT][2];
  bool rise = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (need_mask) {
        const int vis = min(nvalid - 1, row_last[nt][j] - cw0);  // last visible slice index
        const int low = kScores ? row_lo[nt][j] - cw0 : 0;       // first one
        if (g > vis || (kScores && g < low)) z[nt][j] = kNegInf;
        if (g + 8 > vis || (kScores && g + 8 < low)) z[nt][2 + j] = kNegInf;
      }
      lmax[nt][j] = fmaxf(z[nt][j], z[nt][2 + j]);
      rise |= lmax[nt][j] > m[nt][j] + tau;  // also true for the first finite maximum
    }
  }
  probs();
  if (__any_sync(kFull, rise)) {
    const bool exact = C::KI8 && __any_sync(kFull, large);
    const float tau_w = exact ? 0.f : kTau, below = exact ? 0.f : kBelowMax;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float tmax = lmax[nt][j];
        tmax = fmaxf(tmax, __shfl_xor_sync(kFull, tmax, 4));
        tmax = fmaxf(tmax, __shfl_xor_sync(kFull, tmax, 8));
        tmax = fmaxf(tmax, __shfl_xor_sync(kFull, tmax, 16));
        if (tmax > m[nt][j] + tau_w) {
          const float top = tmax - below;
          const float alpha = fast_exp2(m[nt][j] - top);  // 0 from the finite start
          m[nt][j] = top;
          l[nt][j] *= alpha;
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            o[mt][nt][j] *= alpha;
            o[mt][nt][2 + j] *= alpha;
          }
        }
      }
    }
    probs();
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) l[nt][j] += p[nt][j] + p[nt][2 + j];

  };

  // o += V^T . P^T for one stage
  // (scored: cells below nlow, which no row sees, may hold anything too)
  auto pv = [&](int s, int nvalid, int nlow, const float (&p)[NT][4], const uint32_t (&vw)[2][VSW]) {
    const uint32_t st = sbase + s * C::STAGE_B;
  // ---------------- O^T += V^T . P^T ----------------
  if constexpr (FMT == KVQ_F16) {
    uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t h01, l01, h23, l23;
      split_pair(p[nt][0], p[nt][1], h01, l01);
      split_pair(p[nt][2], p[nt][3], h23, l23);
      if constexpr (HL) {  // columns 0-3 hi, 4-7 lo
        bh[nt][0] = movmatrix_t(t >= 2 ? l01 : h01);
        bh[nt][1] = movmatrix_t(t >= 2 ? l23 : h23);
      } else {
        bh[nt][0] = movmatrix_t(h01);
        bh[nt][1] = movmatrix_t(h23);
        bl[nt][0] = movmatrix_t(l01);
        bl[nt][1] = movmatrix_t(l23);
      }
    }
    // V rows of cells past the valid ones may hold anything: zero them.
    const auto keeps = [&](int i) -> bool { return i < nvalid && (!kScores || i >= nlow); };
    const uint32_t mlo = (keeps(2 * t) ? 0xffffu : 0u) | (keeps(2 * t + 1) ? 0xffff0000u : 0u);
    const uint32_t mhi = (keeps(2 * t + 8) ? 0xffffu : 0u) | (keeps(2 * t + 9) ? 0xffff0000u : 0u);
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      uint32_t af[4];
      ldsm_x4_t(af, st + vx[mt & 3] + (uint32_t)(mt >> 2) * kSpanB);
      if (nvalid < kCellsPerWarp || (kScores && nlow > 0)) {
        af[0] &= mlo;
        af[1] &= mlo;
        af[2] &= mhi;
        af[3] &= mhi;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma16816(o[mt][nt], af, bh[nt][0], bh[nt][1]);
        if constexpr (!HL) mma16816(o[mt][nt], af, bl[nt][0], bl[nt][1]);
      }
    }
  } else if constexpr (C::V4) {
    uint32_t sw[2][VSW];
#pragma unroll
    for (int ci = 0; ci < 2; ++ci)
#pragma unroll
      for (int i = 0; i < VSW; ++i) sw[ci][i] = clamp_finite_h2(vw[ci][i]);
    // One ldmatrix.trans x4 per two 32-dim blocks, on 16-bit units of 4
    // nibbles: register (cells 2t, 2t + 1; unit g) holds dims 4g .. 4g + 3
    // of the block for both cells.  Nibble e of both halves becomes the
    // fp16 pair (code - 8) exactly (OR into 1024's exponent, then minus
    // 1032; for the upper nibble of a byte 1024 + 16 code, times 1/16,
    // minus 72), and the block's scales are folded into P (fp32, then the
    // hi + lo split), as the int8 path does per 64-dim group.  Nibbles are
    // always finite and masked cells have p = 0, so no V mask is needed;
    // a masked cell's scale bits may be anything, and clamping them to
    // +-65504 keeps 0 * s == 0 (finite scales pass unchanged).
    // M-tile 2 blk + h: row g is dim 32 blk + 4g + 2h, row g + 8 the dim
    // after it.
#pragma unroll
    for (int kq = 0; kq < C::VROWB / 32; ++kq) {
      uint32_t r[4];
      ldsm_x4_t(r, st + vq[kq]);
#pragma unroll
      for (int jb = 0; jb < 2; ++jb) {
        const int blk = 2 * kq + jb;
        const int sh = 16 * (blk & 1);
        const float s0 = __half2float(__ushort_as_half((unsigned short)(sw[0][blk >> 1] >> sh)));
        const float s8 = __half2float(__ushort_as_half((unsigned short)(sw[1][blk >> 1] >> sh)));
        uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t h01, l01, h23, l23;
          split_pair(p[nt][0] * s0, p[nt][1] * s0, h01, l01);
          split_pair(p[nt][2] * s8, p[nt][3] * s8, h23, l23);
          if constexpr (HL) {
            bh[nt][0] = movmatrix_t(t >= 2 ? l01 : h01);
            bh[nt][1] = movmatrix_t(t >= 2 ? l23 : h23);
          } else {
            bh[nt][0] = movmatrix_t(h01);
            bh[nt][1] = movmatrix_t(h23);
            bl[nt][0] = movmatrix_t(l01);
            bl[nt][1] = movmatrix_t(l23);
          }
        }
        const uint32_t wl = r[2 * jb], wh = r[2 * jb + 1];
        const uint32_t wl8 = wl >> 8, wh8 = wh >> 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t xl = h ? wl8 : wl, xh = h ? wh8 : wh;
          const uint32_t af[4] = {nib_lo(xl), nib_hi(xl), nib_lo(xh), nib_hi(xh)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(o[2 * blk + h][nt], af, bh[nt][0], bh[nt][1]);
            if constexpr (!HL) mma16816(o[2 * blk + h][nt], af, bl[nt][0], bl[nt][1]);
          }
        }
      }
    }
  } else {
    // p = 0 exactly for masked cells, whose scale bits may be anything
    // (even +-inf / NaN): clamping to +-65504 keeps 0 * s == 0.  Finite
    // fp16 scales pass unchanged.
    uint32_t sw[2][VSW];
#pragma unroll
    for (int ci = 0; ci < 2; ++ci)
#pragma unroll
      for (int i = 0; i < VSW; ++i) sw[ci][i] = clamp_finite_h2(vw[ci][i]);
#pragma unroll
    for (int gv = 0; gv < C::NG; ++gv) {
      const float s0 = gv & 1 ? half_hi(sw[0][gv >> 1]) : half_lo(sw[0][gv >> 1]);
      const float s8 = gv & 1 ? half_hi(sw[1][gv >> 1]) : half_lo(sw[1][gv >> 1]);
      uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float x0 = p[nt][0] * s0;
        const float x1 = p[nt][1] * s0;
        const float x2 = p[nt][2] * s8;
        const float x3 = p[nt][3] * s8;
        uint32_t h01, l01, h23, l23;
        split_pair(x0, x1, h01, l01);
        split_pair(x2, x3, h23, l23);
        if constexpr (HL) {
          bh[nt][0] = movmatrix_t(t >= 2 ? l01 : h01);
          bh[nt][1] = movmatrix_t(t >= 2 ? l23 : h23);
        } else {
          bh[nt][0] = movmatrix_t(h01);
          bh[nt][1] = movmatrix_t(h23);
          bl[nt][0] = movmatrix_t(l01);
          bl[nt][1] = movmatrix_t(l23);
        }
      }
      // Two ldmatrix.trans x4 per 64-dim group, on byte pairs: register
      // i of chunk c holds (cell 2t, dims 16c + 2g, +1) and (cell 2t + 1,
      // same dims) for cells +0 (i = 0) or +8 (i = 1), so m-tile c row g is
      // dim 16c + 2g and row g + 8 is dim 16c + 2g + 1.
#pragma unroll
      for (int jh = 0; jh < 2; ++jh) {
        const int c0 = gv * 4 + jh * 2;  // first 16-dim chunk of this pair
        uint32_t r[4];
        ldsm_x4_t(r, st + C::OFF_V + kstep(c0 >> 1));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w0 = r[2 * h] ^ 0x80808080u, w8 = r[2 * h + 1] ^ 0x80808080u;
          uint32_t af[4];
          af[0] = hsub2(prmt(w0, kMagic, 0x4240u), kBias);  // dim 2g, cells 2t, 2t+1
          af[1] = hsub2(prmt(w0, kMagic, 0x4341u), kBias);  // dim 2g+1
          af[2] = hsub2(prmt(w8, kMagic, 0x4240u), kBias);  // dim 2g, cells 2t+8, 2t+9
          af[3] = hsub2(prmt(w8, kMagic, 0x4341u), kBias);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(o[c0 + h][nt], af, bh[nt][0], bh[nt][1]);
            if constexpr (!HL) mma16816(o[c0 + h][nt], af, bl[nt][0], bl[nt][1]);
          }
        }
      }
    }
  }
  };

  auto release = [&](int it) {
    // the last warp to let the stage go issues its refill
    __syncwarp();
    if constexpr (kSlices) {   // (its own slice: every lane's reads are done)
      if (it + C::STAGES < n_tiles) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        issue_slice(it + C::STAGES, blk_in_smem);
      }
      return;
    }
    if constexpr (kScores) {
      const int s = it % C::STAGES;
      int prev = 0;
      if (lane == 0) {
        asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;"
                     : "=r"(prev)
                     : "r"(smem_u32(s_rel + s))
                     : "memory");
        if (prev == kConsumerWarps - 1) s_rel[s] = 0;
      }
      prev = __shfl_sync(kFull, prev, 0);
      if (prev == kConsumerWarps - 1 && it + C::STAGES < n_tiles) {
        __syncwarp();   // (lane 0's acquire holds for the lanes that issue)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        issue_warp(it + C::STAGES, blk_in_smem);
      }
      return;
    }
    if (lane == 0) {
      const int s = it % C::STAGES;
      // acquire-release: this warp's reads of the stage happen before the
      // count moves, and the last warp sees every other warp's reads done
      int prev;
      asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;"
                   : "=r"(prev)
                   : "r"(smem_u32(s_rel + s))
                   : "memory");
      if (prev == kConsumerWarps - 1) {
        s_rel[s] = 0;
        if (it + C::STAGES < n_tiles) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          int nb[MAXP];
          tile_blks(it + C::STAGES, blk_in_smem, nb);
          issue(it + C::STAGES, nb);
        }
      }
    }
  };

  // Software pipeline: q.k of tile it+1 and p.v of tile it form one
  // straight-line block, so the compiler can interleave the two; the
  // softmax of tile it+1 follows because it may rescale o.  Neither is
  // skipped for a slice without valid cells (stale or unloaded stage
  // memory): its logits are masked to -inf, so p = 0, FP16 V rows are
  // zeroed by mask and int8 V scales are clamped to finite values.
  int blk_n = slice_blk(0);
  int nv_cur = 0;
  float p_cur[NT][4];
  uint32_t vw[2][VSW];   // V scales of the tile whose p.v comes next
  if (n_tiles > 0) {
    if (!mbar_wait(bar_own, 0, a.wait_limit)) {
      lost = true;
    } else {
      nv_cur = slice_nvalid(0, blk_n);
      blk_n = slice_blk(1);
      load_scales(0, vw);
      float z[NT][4];
      qk(0, z);
      softmax(nv_cur, c_begin + tile_of(0) * kTC + cl, vw, z, p_cur);
    }
  }
  int it = 0;
  for (; it + 1 < n_tiles && !lost; ++it) {
    const int sn = (it + 1) % C::STAGES;
    if (!mbar_wait(bar_own + 8 * sn, ((it + 1) / C::STAGES) & 1, a.wait_limit)) {
      lost = true;
      break;
    }
    const int nv_next = slice_nvalid(it + 1, blk_n);
    blk_n = slice_blk(it + 2);
    uint32_t vn[2][VSW];
    load_scales(sn, vn);
    float zn[NT][4];
    qk(sn, zn);
    pv(it % C::STAGES, nv_cur, lo_all - (c_begin + tile_of(it) * kTC + cl), p_cur, vw);
    release(it);
    softmax(nv_next, c_begin + tile_of(it + 1) * kTC + cl, vn, zn, p_cur);
    nv_cur = nv_next;
#pragma unroll
    for (int i = 0; i < 2 * VSW; ++i) vw[i / VSW][i % VSW] = vn[i / VSW][i % VSW];
  }
  if (!lost && n_tiles > 0) {  // the last tile
    pv(it % C::STAGES, nv_cur, lo_all - (c_begin + tile_of(it) * kTC + cl), p_cur, vw);
    release(it);
  }
  if (kSlices ? lane == 0 : producer) {
    // Every copy this CTA issued (kSlices: this warp) has landed before the CTA
    // can exit (waits return at once in normal runs; they are bounded after a
    // lost wait).
    const int n_all = n_tiles > n_first ? n_tiles : n_first;
    for (int it = n_all > C::STAGES ? n_all - C::STAGES : 0; it < n_all; ++it)
      (void)mbar_wait(bar_own + 8 * (it % C::STAGES), (it / C::STAGES) & 1, a.wait_limit);
  }

  // ---------------- merge the 4 warps, write the split's partial ----------------
  // Each warp's row maxima and sums go to shared memory; after one barrier
  // (every warp is past the loop, so the stages are free) each warp writes
  // its rows scaled to the CTA maximum into a slab of its own in the stage
  // memory; after a second barrier the 4 slabs are summed straight into the
  // split's partial in global memory.  A lost wait poisons the rows (NaN).
  if constexpr (HL) {
    // the hi and lo column sums of each row meet (lanes t < 2 keep them)
#pragma unroll
    for (int mt = 0; mt < KS; ++mt)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[mt][0][k] += __shfl_xor_sync(kFull, o[mt][0][k], 2);
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float v = l[nt][j];
      v += __shfl_xor_sync(kFull, v, 4);
      v += __shfl_xor_sync(kFull, v, 8);
      v += __shfl_xor_sync(kFull, v, 16);
      l[nt][j] = v;
    }
  float* s_wml = reinterpret_cast<float*>(smem + C::SMEM_WML);  // [warp][RP][m, l]
  const bool wlost = __any_sync(kFull, lost);
  if (g == 0 && (!HL || t < 2)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = row_of(nt, j);
        s_wml[(warp * RP + r) * 2 + 0] = wlost ? __int_as_float(0x7fc00000) : m[nt][j];
        s_wml[(warp * RP + r) * 2 + 1] = l[nt][j];
      }
  }
  __syncthreads();
  float* s_slab = reinterpret_cast<float*>(smem);  // [warp][R][HD] over the free stages
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = row_of(nt, j);
      if (r < Rc && (!HL || t < 2)) {
        float M = s_wml[r * 2];
#pragma unroll
        for (int w = 1; w < kConsumerWarps; ++w) M = fmaxf(M, s_wml[(w * RP + r) * 2]);
        const float wgt = (M == kNegInf || m[nt][j] == kNegInf) ? 0.f : fast_exp2(m[nt][j] - M);
        float* orow = s_slab + (warp * Rc + r) * HD;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          if constexpr (FMT == KVQ_F16) {  // m-tile rows g, g + 8 are dims 16 mt + g, + 8
            orow[mt * 16 + g] = wgt * o[mt][nt][j];
            orow[mt * 16 + g + 8] = wgt * o[mt][nt][2 + j];
          } else if constexpr (C::V4) {   // K8V4: dims 32 (mt / 2) + 4g + 2 (mt % 2), + 1
            *reinterpret_cast<float2*>(orow + (mt >> 1) * 32 + 4 * g + 2 * (mt & 1)) =
                make_float2(wgt * o[mt][nt][j], wgt * o[mt][nt][2 + j]);
          } else {                        // int8: dims 16 mt + 2g, + 1
            *reinterpret_cast<float2*>(orow + mt * 16 + 2 * g) =
                make_float2(wgt * o[mt][nt][j], wgt * o[mt][nt][2 + j]);
          }
        }
      }
    }
  __syncthreads();
  if constexpr (kLists) {
    if (clustered) {
      merge_cluster<FMT, HD, NT>(a, smem, b, r0, Rc);
      return;
    }
  }
  // this CTA's rows of the split's partial
  const size_t row0 = (kScores && a.batch_items > 0 ? (size_t)kvh * a.batch_items + slot
                                                    : ((size_t)b * a.n_kv + kvh) * a.nsplit + split) * a.R + r0;
  if constexpr (C::V4) {
    // K8V4: the merged rows are in the rotated basis; one warp per row sums
    // the slabs, rotates the row back (Walsh-Hadamard, divided by HD) and
    // writes it.  The combine is linear in the partials, so it needs no
    // change.
    constexpr int U = HD >= 128 ? 4 : 2, NI = HD / (32 * U);
    for (int r = warp; r < Rc; r += kConsumerWarps) {
      float x[NI][U];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int d0 = U * lane + 32 * U * i;
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const float* col = s_slab + r * HD + d0 + e;
          x[i][e] = (col[0] + col[Rc * HD]) + (col[2 * Rc * HD] + col[3 * Rc * HD]);
        }
      }
      wht_warp<U, NI>(x, lane);
      float* dst = a.ws_o + (row0 + r) * HD;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int d0 = U * lane + 32 * U * i;
        if constexpr (U == 4)
          *reinterpret_cast<float4*>(dst + d0) =
              make_float4(x[i][0] * (1.0f / HD), x[i][1] * (1.0f / HD), x[i][U > 2 ? 2 : 0] * (1.0f / HD),
                          x[i][U > 3 ? 3 : 0] * (1.0f / HD));
        else
          *reinterpret_cast<float2*>(dst + d0) = make_float2(x[i][0] * (1.0f / HD), x[i][1] * (1.0f / HD));
      }
    }
  } else
  for (int i4 = threadIdx.x; i4 < Rc * HD / 4; i4 += kThreads) {
    const float4 v0 = reinterpret_cast<const float4*>(s_slab)[i4];
    const float4 v1 = reinterpret_cast<const float4*>(s_slab + Rc * HD)[i4];
    const float4 v2 = reinterpret_cast<const float4*>(s_slab + 2 * Rc * HD)[i4];
    const float4 v3 = reinterpret_cast<const float4*>(s_slab + 3 * Rc * HD)[i4];
    reinterpret_cast<float4*>(a.ws_o + row0 * HD)[i4] =
        make_float4((v0.x + v1.x) + (v2.x + v3.x), (v0.y + v1.y) + (v2.y + v3.y),
                    (v0.z + v1.z) + (v2.z + v3.z), (v0.w + v1.w) + (v2.w + v3.w));
  }
  if (threadIdx.x < Rc) {
    const int r = threadIdx.x;
    float M = s_wml[r * 2];
    bool bad = M != M;
#pragma unroll
    for (int w = 1; w < kConsumerWarps; ++w) {
      const float mw = s_wml[(w * RP + r) * 2];
      bad |= mw != mw;
      M = fmaxf(M, mw);
    }
    float lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kConsumerWarps; ++w) {
      const float mw = s_wml[(w * RP + r) * 2];
      if (M != kNegInf && mw != kNegInf) lsum = fmaf(s_wml[(w * RP + r) * 2 + 1], fast_exp2(mw - M), lsum);
    }
    *reinterpret_cast<float2*>(a.ws_ml + (row0 + r) * 2) =
        make_float2(bad ? __int_as_float(0x7fc00000) : M, lsum);
  }
}

// ---------------------------------------------------------------------------
// Final combine of the per-warp partials, launched as a programmatic
// dependent of the partial kernel: its CTAs wait on griddepcontrol until
// every partial is written.
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 256;
constexpr int kCombineBatch = 4;   // partial loads in flight per thread

template <int HD, int DV>
__global__ void __launch_bounds__(kCombineThreads, 4) combine_partials(DecodeArgs a) {
  // One CTA per (KV head, sequence, row, DV float4 columns).  Thread (js,
  // dv) merges column dv of the partials j = js, js + JS, ... online
  // (running maximum, rescaled sums; the loads of a batch issued together);
  // the JS slices then meet through warp shuffles and shared memory.  The
  // host picks DV so that one batch usually covers every partial.
  constexpr int JS = kCombineThreads / DV;
  constexpr int NW = kCombineThreads / 32;
  constexpr int CHUNKS = HD / 4 / DV;   // CTAs per row
  constexpr float kNegInf = -INFINITY;
  static_assert(DV <= 32 && HD / 4 % DV == 0, "combine shape");
  __shared__ float s_wm[NW];
  __shared__ float s_wl[NW];
  __shared__ int s_wbad[NW];
  __shared__ float4 s_wacc[NW][DV];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // (block lists: the grid's x runs over the lists, which may exceed y's limit)
  const int kvh = kLists ? 0 : blockIdx.x, b = kLists ? blockIdx.x : blockIdx.y;
  const int r = blockIdx.z / CHUNKS, d0 = (blockIdx.z % CHUNKS) * DV * 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int dv = tid % DV, js = tid / DV;
  const int d = d0 + 4 * dv;
  // one sequence: every split slot is written (splits past the context say
  // "no cells"), so the context length need not be read
  int nlive = a.nsplit;
  size_t base0 = ((size_t)b * a.n_kv + kvh) * a.nsplit;
  if (kScores && a.batch_items > 0) {
    const int first = __ldcg(a.ws_base + b);
    nlive = __ldcg(a.ws_base + b + 1) - first;
    base0 = (size_t)kvh * a.batch_items + first;
  } else if (kLists || a.n_seq > 1) {
    const Span sp = span_of(a, b, __ldg(a.ctx_lens + b));
    nlive = (int)fdiv((unsigned)(sp.end - sp.base + a.split_cells - 1), a.div_split);
  }

  float M = kNegInf, lsum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  bool bad = false;
  for (int j0 = js; j0 < nlive; j0 += JS * kCombineBatch) {
    float mb[kCombineBatch], lb[kCombineBatch];
    float4 ob[kCombineBatch];
#pragma unroll
    for (int u = 0; u < kCombineBatch; ++u) {
      const int j = j0 + u * JS;
      mb[u] = kNegInf;
      lb[u] = 0.f;
      ob[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < nlive) {
        const size_t rj = (base0 + j) * a.R + r;
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.ws_ml + rj * 2));
        mb[u] = ml.x;
        lb[u] = ml.y;
        ob[u] = __ldcg(reinterpret_cast<const float4*>(a.ws_o + rj * HD + d));
      }
    }
    float bm = M;
#pragma unroll
    for (int u = 0; u < kCombineBatch; ++u) {
      bad |= mb[u] != mb[u];
      bm = fmaxf(bm, mb[u]);
    }
    if (bm == kNegInf) continue;
    const float sc = M == kNegInf ? 0.f : fast_exp2(M - bm);
    acc.x *= sc;
    acc.y *= sc;
    acc.z *= sc;
    acc.w *= sc;
    lsum *= sc;
#pragma unroll
    for (int u = 0; u < kCombineBatch; ++u) {
      if (mb[u] != kNegInf) {
        const float w = fast_exp2(mb[u] - bm);
        acc.x = fmaf(w, ob[u].x, acc.x);
        acc.y = fmaf(w, ob[u].y, acc.y);
        acc.z = fmaf(w, ob[u].z, acc.z);
        acc.w = fmaf(w, ob[u].w, acc.w);
        lsum = fmaf(w, lb[u], lsum);
      }
    }
    M = bm;
  }
  // block maximum (a warp holds 32 / DV slices; their columns share M)
  float wm = M;
#pragma unroll
  for (int off = DV; off < 32; off <<= 1) wm = fmaxf(wm, __shfl_xor_sync(kFull, wm, off));
  const bool wbad = __any_sync(kFull, bad);
  if (lane == 0) {
    s_wm[warp] = wm;
    s_wbad[warp] = wbad;
  }
  __syncthreads();
  float Mall = s_wm[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) Mall = fmaxf(Mall, s_wm[w]);
  const float sc = (M == kNegInf || Mall == kNegInf) ? 0.f : fast_exp2(M - Mall);
  acc.x *= sc;
  acc.y *= sc;
  acc.z *= sc;
  acc.w *= sc;
  lsum *= sc;
#pragma unroll
  for (int off = DV; off < 32; off <<= 1) {
    acc.x += __shfl_xor_sync(kFull, acc.x, off);
    acc.y += __shfl_xor_sync(kFull, acc.y, off);
    acc.z += __shfl_xor_sync(kFull, acc.z, off);
    acc.w += __shfl_xor_sync(kFull, acc.w, off);
    lsum += __shfl_xor_sync(kFull, lsum, off);
  }
  if (lane < DV) s_wacc[warp][lane] = acc;
  if (lane == 0) s_wl[warp] = lsum;
  __syncthreads();
  if (tid < DV) {
    float4 sum = s_wacc[0][tid];
    float lam = s_wl[0];
    int any_bad = s_wbad[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const float4 v = s_wacc[w][tid];
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
      lam += s_wl[w];
      any_bad |= s_wbad[w];
    }
    // an empty context (no live partial) gives 0; a lost wait gives NaN
    const float inv = lam > 0.f ? 1.f / lam : 0.f;
    float4 res = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
    if (any_bad) {
      const float nan = __int_as_float(0x7fc00000);
      res = make_float4(nan, nan, nan, nan);
    }
    const int w = div_g(a, r), gg = r - w * a.G;
    *reinterpret_cast<float4*>(a.out + (((size_t)b * a.W + w) * a.n_q + (size_t)kvh * a.G + gg) * HD +
                               d0 + 4 * tid) = res;
  }
}

template <int HD, int DV>
cudaError_t launch_combine_dv(const DecodeArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cc = {};
  cc.gridDim = kLists ? dim3(a.n_seq, 1, a.R * (HD / 4 / DV)) : dim3(a.n_kv, a.n_seq, a.R * (HD / 4 / DV));
  cc.blockDim = dim3(kCombineThreads);
  cc.stream = s;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cc.attrs = pdl;
  cc.numAttrs = 1;
  return cudaLaunchKernelEx(&cc, combine_partials<HD, DV>, a);
}

// Widest column block (fewest CTAs) whose slices still cover every partial
// slot in one batch of loads; 4 columns (64 slices) when none does.
template <int HD>
cudaError_t launch_combine(const DecodeArgs& a, cudaStream_t s) {
  const int most = kScores && a.batch_items > 0 ? a.batch_items / a.n_seq + 1 : a.nsplit;   // (a batch's mean)
  const int need_js = (most + kCombineBatch - 1) / kCombineBatch;
  constexpr int MAXDV = HD / 4 < 32 ? HD / 4 : 32;
  if (need_js <= kCombineThreads / 32 && MAXDV >= 32) return launch_combine_dv<HD, MAXDV>(a, s);
  if (need_js <= kCombineThreads / 16 && MAXDV >= 16) return launch_combine_dv<HD, 16>(a, s);
  if (need_js <= kCombineThreads / 8) return launch_combine_dv<HD, 8>(a, s);
  return launch_combine_dv<HD, 4>(a, s);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
}

// Span sp of one codes array: [total rows][span bytes] starting at byte
// sp * span of each row (rows of row_bytes), box = one piece of cells, the
// swizzle as wide as the span (32, 64 or 128 bytes).
bool make_map(CUtensorMap* map, const void* base, int span, int row_bytes, int sp, long long rows,
              int piece_cells) {
  auto enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)span, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {(cuuint32_t)span, (cuuint32_t)piece_cells};
  const cuuint32_t estr[2] = {1, 1};
  void* span_base = static_cast<char*>(const_cast<void*>(base)) + (size_t)sp * span;
  const CUtensorMapSwizzle sw = span == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                : span == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                             : CU_TENSOR_MAP_SWIZZLE_32B;
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, span_base, dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Resident CTAs per SM of one configuration (0 if it cannot run), after
// raising its dynamic shared-memory limit; done once per context.
template <int FMT, int HD, int NT, bool HL>
int ctas_per_sm_impl() {
  static ContextCache<int> cache;
  int occ = 0;
  const bool ok = per_context(cache, &occ, [](int* v) {
    using C = Cfg<FMT, HD, NT>;
    if (cudaFuncSetAttribute(decode_mma<FMT, HD, NT, HL>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
      return false;
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, decode_mma<FMT, HD, NT, HL>, kThreads,
                                                      C::SMEM) != cudaSuccess)
      return false;
    *v = n;
    return true;
  });
  return ok ? occ : 0;
}

template <int FMT, int HD, int NT, bool HL>
cudaError_t launch_impl(const DecodePlan& p, const DecodeArgs& a, cudaStream_t s) {
  using C = Cfg<FMT, HD, NT>;
  if (ctas_per_sm_impl<FMT, HD, NT, HL>() <= 0) return cudaErrorInvalidConfiguration;
  const long long rows = (long long)a.pool.n_blocks * a.pool.n_kv << a.pool.bs_log2;
  const int piece = kWarpSlices<HD, HL> ? kCellsPerWarp : 1 << (a.pool.bs_log2 < 6 ? a.pool.bs_log2 : 6);
  TmaMaps maps;
  memset(&maps, 0, sizeof(maps));
  for (int sp = 0; sp < C::NCH; ++sp)
    if (!make_map(&maps.k[sp], a.pool.k, C::SWB, C::ROWB, sp, rows, piece)) return cudaErrorInvalidValue;
  for (int sp = 0; sp < C::VNCH; ++sp)
    if (!make_map(&maps.v[sp], a.pool.v, C::VSWB, C::VROWB, sp, rows, piece)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  const long long items =
      kScores && a.batch_items > 0 ? (long long)a.batch_items * a.n_kv * a.n_rt : (long long)p.nsplit * a.n_kv * a.n_seq * a.n_rt;
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)items);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (kLists && a.c_log2 >= 0) {   // no partials, no combine
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1u << a.c_log2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, decode_mma<FMT, HD, NT, HL>, maps, a);
  }
  cudaError_t e = cudaLaunchKernelEx(&cfg, decode_mma<FMT, HD, NT, HL>, maps, a);
  if (e != cudaSuccess) return e;
  return launch_combine<HD>(a, s);
}

// Kernel shape of a row count: 0 = one 8-column tile with hi/lo columns
// (at most 4 rows), else the number of 8-row tiles.
int tile_code(int rows) { return rows <= 4 ? 0 : rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : -1; }

template <int FMT, int HD>
int ctas_per_sm_hd(int code) {
  switch (code) {
    case 0: return ctas_per_sm_impl<FMT, HD, 1, true>();
    case 1: return ctas_per_sm_impl<FMT, HD, 1, false>();
    case 2: if constexpr (HD <= 128 || kScores) return ctas_per_sm_impl<FMT, HD, 2, false>(); break;
    case 4: if constexpr (HD <= 64) return ctas_per_sm_impl<FMT, HD, 4, false>(); break;
  }
  return 0;
}

template <int FMT, int HD>
cudaError_t launch_hd(int code, const DecodePlan& p, const DecodeArgs& a, cudaStream_t s) {
  switch (code) {
    case 0: return launch_impl<FMT, HD, 1, true>(p, a, s);
    case 1: return launch_impl<FMT, HD, 1, false>(p, a, s);
    case 2: if constexpr (HD <= 128 || kScores) return launch_impl<FMT, HD, 2, false>(p, a, s); break;
    case 4: if constexpr (HD <= 64) return launch_impl<FMT, HD, 4, false>(p, a, s); break;
  }
  return cudaErrorInvalidValue;
}

}  // namespace

#if !KVQ_DECODE_LISTS && !KVQ_DECODE_SCORES

void* tensor_map_encoder() {
  static void* fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = f;
  });
  return fn;
}

unsigned long long current_context_id() {
  using GetCurrent = CUresult (*)(CUcontext*);
  using GetId = CUresult (*)(CUcontext, unsigned long long*);
  static GetCurrent get_current = nullptr;
  static GetId get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<GetCurrent>(f);
    f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<GetId>(f);
    (void)cudaGetLastError();
  });
  if (get_current == nullptr || get_id == nullptr) return 0;
  CUcontext ctx = nullptr;
  if (get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return 0;
  unsigned long long id = 0;
  if (get_id(ctx, &id) != CUDA_SUCCESS) return 0;
  return id;
}

bool mma_decode_supported(int fmt, int hd, int rows) {
  if (rows < 1 || rows > 32) return false;
  if (hd != 64 && hd != 128 && hd != 256) return false;
  return fmt == KVQ_F16 || fmt == KVQ_Q8 || fmt == KVQ_K8V4;
}

// Query rows one CTA holds: 8-row MMA tiles while their fp32 accumulators
// (HD / 16 m-tiles x 4 floats per tile and thread) stay at 32 per thread
// or fewer -- 32 rows at head_dim 64, 16 at 128, 8 at 256.
int mma_rows_per_cta(int hd) { return 8 * (256 / hd); }
// Scored: 16 at 256 too, twice the accumulators, but half of the widening and of
// the copies a row (2 x 98000 cells, 2 heads, 32 rows of 256 dims, blocks of 16 /
// 256: FP16 194 / 146 -> 155 / 131 us, int8 137 / 118 -> 112 / 101, K8V4 129 / 116 ->
// 122 / 110).
int scores_rows_per_cta(int hd) { return hd == 256 ? 16 : mma_rows_per_cta(hd); }

int mma_cell_tile() { return kTC; }

#endif  // the dense decode

#if KVQ_DECODE_LISTS
#define KVQ_CTAS_PER_SM lists_ctas_per_sm
#define KVQ_LAUNCH launch_decode_lists
#elif KVQ_DECODE_SCORES
#define KVQ_CTAS_PER_SM scores_ctas_per_sm
#define KVQ_LAUNCH launch_decode_scores
#else
#define KVQ_CTAS_PER_SM mma_ctas_per_sm
#define KVQ_LAUNCH launch_decode_mma_partial
#endif

int KVQ_CTAS_PER_SM(int fmt, int hd, int rows) {
  const int nt = tile_code(rows);
  if (fmt == KVQ_F16) {
    if (hd == 64) return ctas_per_sm_hd<KVQ_F16, 64>(nt);
    if (hd == 128) return ctas_per_sm_hd<KVQ_F16, 128>(nt);
    return ctas_per_sm_hd<KVQ_F16, 256>(nt);
  }
  if (fmt == KVQ_Q8) {
    if (hd == 64) return ctas_per_sm_hd<KVQ_Q8, 64>(nt);
    if (hd == 128) return ctas_per_sm_hd<KVQ_Q8, 128>(nt);
    return ctas_per_sm_hd<KVQ_Q8, 256>(nt);
  }
  if (hd == 64) return ctas_per_sm_hd<KVQ_K8V4, 64>(nt);
  if (hd == 128) return ctas_per_sm_hd<KVQ_K8V4, 128>(nt);
  return ctas_per_sm_hd<KVQ_K8V4, 256>(nt);
}

cudaError_t KVQ_LAUNCH(int fmt, int hd, const DecodePlan& p, const DecodeArgs& a, cudaStream_t s) {
  const int nt = tile_code(p.rt_rows);
  if (fmt == KVQ_F16) {
    if (hd == 64) return launch_hd<KVQ_F16, 64>(nt, p, a, s);
    if (hd == 128) return launch_hd<KVQ_F16, 128>(nt, p, a, s);
    return launch_hd<KVQ_F16, 256>(nt, p, a, s);
  }
  if (fmt == KVQ_Q8) {
    if (hd == 64) return launch_hd<KVQ_Q8, 64>(nt, p, a, s);
    if (hd == 128) return launch_hd<KVQ_Q8, 128>(nt, p, a, s);
    return launch_hd<KVQ_Q8, 256>(nt, p, a, s);
  }
  if (hd == 64) return launch_hd<KVQ_K8V4, 64>(nt, p, a, s);
  if (hd == 128) return launch_hd<KVQ_K8V4, 128>(nt, p, a, s);
  return launch_hd<KVQ_K8V4, 256>(nt, p, a, s);
}

}  // namespace kvq
