// kvq_bounds.cu -- bounds of each cache block's keys (kvq_bound_blocks).
//
// For a block's live cells and one KV head, lo[d] = min and hi[d] = max over
// the cells of the dequantised key K[c][d]; per 64 dims, s = 2^e with the
// smallest e in [-24, 16] that gives 127 s >= max(|lo|, |hi|), and the codes
// floor(lo / s) and ceil(hi / s).  All of it is exact: the dequantised keys
// are fp16 values or products of an int8 code and an fp16 scale, which fp32
// holds exactly, and a division by a power of two does not round.
//
// A work item is one (block, KV head): block_size contiguous rows of K.
// Its warps read them with 16-byte loads, each lane always at the same
// dims, keep the running minima and maxima in registers and meet at the end
// (shuffles between the lanes of one dim, shared memory between warps).
// Bound by the read of K.
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kBoundThreads = 256;
constexpr unsigned kAll = 0xffffffffu;

// The smallest e with 127 * 2^e >= m (m >= 0, finite or inf), in [lowest, highest].
__device__ __forceinline__ int scale_exponent(float m, int lowest, int highest) {
  const uint32_t b = __float_as_uint(m);
  const int x = (int)(b >> 23) - 126;                     // m = f 2^x, f in [1/2, 1) (normal m)
  const int e = x - 7 + ((b & 0x7fffffu) > 0x7e0000u);    // f > 127/128
  return min(max(e, lowest), highest);                    // (0 and subnormals: lowest)
}

__device__ __forceinline__ float pow2f_exact(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// FMT: KVQ_F16, or KVQ_Q8 for both int8-K formats.  WPI warps per item.
template <int FMT, int HD, int WPI>
__global__ void __launch_bounds__(kBoundThreads) bound_blocks_kernel(BoundArgs a) {
  constexpr bool I8 = FMT != KVQ_F16;
  constexpr int VD = I8 ? 16 : 8;         // dims per 16-byte load
  constexpr int LPR = HD / VD;            // lanes per row
  constexpr int RPW = 32 / LPR;           // rows a warp reads at once
  constexpr int NG = HD / kGroup;
  constexpr int ITEMS = kBoundThreads / 32 / WPI;   // items per CTA
  constexpr int LG = kGroup / VD;         // lanes of one 64-dim group
  __shared__ float s_red[WPI > 1 ? WPI : 1][2][HD];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31;
  const int wi = (tid >> 5) % WPI;        // warp within its item
  const long long item = (long long)blockIdx.x * ITEMS + (tid >> 5) / WPI;
  // item = (sequence, touched block, KV head), heads innermost
  const long long sb = item / a.pool.n_kv;
  const int h = (int)(item - sb * a.pool.n_kv);
  const int b = (int)(sb / a.touched), tb = (int)(sb - (long long)b * a.touched);
  int blk = -1, live = 0;
  if (b < a.n_seq) {
    const int bs = 1 << a.pool.bs_log2;
    const long long cap = (long long)a.max_blocks << a.pool.bs_log2;
    const long long len = min((long long)__ldg(a.ctx_lens + b), cap);
    const long long start = a.ctx_start != nullptr ? max(__ldg(a.ctx_start + b), 0) : 0;
    const long long j = (start >> a.pool.bs_log2) + tb;
    if (start < len && (j << a.pool.bs_log2) < len) {
      blk = __ldg(a.block_table + (size_t)b * a.max_blocks + j);
      live = (int)min((long long)bs, len - (j << a.pool.bs_log2));
    }
  }
  const bool has = blk >= 0 && blk < a.pool.n_blocks;
  if (WPI == 1 && !has) return;   // (WPI > 1: every warp of the CTA has the same item)
  if (WPI > 1 && ITEMS == 1 && !has) return;

  const int l = lane % LPR, r0 = wi * RPW + lane / LPR;
  float lo[VD], hi[VD];
#pragma unroll
  for (int e = 0; e < VD; ++e) {
    lo[e] = INFINITY;
    hi[e] = -INFINITY;
  }
  if (has) {
    const size_t row0 = ((size_t)blk * a.pool.n_kv + h) << a.pool.bs_log2;
    if constexpr (!I8) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __half*>(a.pool.k) + row0 * HD) + l;
      __half2 mn[4], mx[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        mn[e] = __halves2half2(__ushort_as_half(0x7c00), __ushort_as_half(0x7c00));
        mx[e] = __halves2half2(__ushort_as_half(0xfc00), __ushort_as_half(0xfc00));
      }
#pragma unroll 8
      for (int r = r0; r < live; r += RPW * WPI) {
        const uint4 u = __ldg(src + (size_t)r * LPR);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 x = *reinterpret_cast<const __half2*>(&w[e]);
          mn[e] = __hmin2(mn[e], x);   // (a NaN operand is passed over)
          mx[e] = __hmax2(mx[e], x);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo[2 * e] = __low2float(mn[e]);
        lo[2 * e + 1] = __high2float(mn[e]);
        hi[2 * e] = __low2float(mx[e]);
        hi[2 * e + 1] = __high2float(mx[e]);
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const int8_t*>(a.pool.k) + row0 * HD) + l;
      const __half* sc = a.pool.ks + row0 * NG + l / LG;
#pragma unroll 4
      for (int r = r0; r < live; r += RPW * WPI) {
        const uint4 u = __ldg(src + (size_t)r * LPR);
        const float s = __half2float(__ldg(sc + (size_t)r * NG));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < VD; ++e) {
          const float x = (float)(int8_t)(w[e / 4] >> (8 * (e % 4))) * s;
          lo[e] = fminf(lo[e], x);
          hi[e] = fmaxf(hi[e], x);
        }
      }
    }
  }
  // the lanes of a warp that hold the same dims
#pragma unroll
  for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
    for (int e = 0; e < VD; ++e) {
      lo[e] = fminf(lo[e], __shfl_xor_sync(kAll, lo[e], off));
      hi[e] = fmaxf(hi[e], __shfl_xor_sync(kAll, hi[e], off));
    }
  if constexpr (WPI > 1) {
    static_assert(ITEMS == 1 || WPI == 1, "one item per CTA when warps share it");
    if (lane < LPR) {
#pragma unroll
      for (int e = 0; e < VD; ++e) {
        s_red[wi][0][l * VD + e] = lo[e];
        s_red[wi][1][l * VD + e] = hi[e];
      }
    }
    __syncthreads();
    if (wi != 0) return;
#pragma unroll
    for (int w = 1; w < WPI; ++w)
#pragma unroll
      for (int e = 0; e < VD; ++e) {
        lo[e] = fminf(lo[e], s_red[w][0][l * VD + e]);
        hi[e] = fmaxf(hi[e], s_red[w][1][l * VD + e]);
      }
  }
  // scale of the 64 dims this lane's belong to (a dim without any number: 0)
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < VD; ++e) {
    if (lo[e] > hi[e]) lo[e] = hi[e] = 0.f;
    m = fmaxf(m, fmaxf(fabsf(lo[e]), fabsf(hi[e])));
  }
#pragma unroll
  for (int off = 1; off < LG; off <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
  const int e2 = scale_exponent(m, -24, 16);
  const float inv = pow2f_exact(-e2);
  uint32_t cl[VD / 4], ch[VD / 4];
#pragma unroll
  for (int i = 0; i < VD / 4; ++i) {
    cl[i] = ch[i] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = max((int)fmaxf(floorf(lo[4 * i + k] * inv), -127.f), -127);
      const int y = min((int)fminf(ceilf(hi[4 * i + k] * inv), 127.f), 127);
      cl[i] |= (uint32_t)(min(x, 127) & 0xff) << (8 * k);
      ch[i] |= (uint32_t)(max(y, -127) & 0xff) << (8 * k);
    }
  }
  if (lane < LPR) {
    int8_t* dst = a.bounds + ((size_t)blk * a.pool.n_kv + h) * 2 * HD + l * VD;
    if constexpr (VD == 16) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(cl[0], cl[1], cl[VD > 8 ? 2 : 0], cl[VD > 8 ? 3 : 0]);
      *reinterpret_cast<uint4*>(dst + HD) = make_uint4(ch[0], ch[1], ch[VD > 8 ? 2 : 0], ch[VD > 8 ? 3 : 0]);
    } else {
      *reinterpret_cast<uint2*>(dst) = make_uint2(cl[0], cl[1]);
      *reinterpret_cast<uint2*>(dst + HD) = make_uint2(ch[0], ch[1]);
    }
    if (l % LG == 0) a.scales[((size_t)blk * a.pool.n_kv + h) * NG + l / LG] = pow2f_exact(e2);
  }
}

template <int FMT, int HD, int WPI>
cudaError_t launch_wpi(const BoundArgs& a, cudaStream_t s) {
  constexpr int ITEMS = kBoundThreads / 32 / WPI;
  const long long items = (long long)a.n_seq * a.touched * a.pool.n_kv;
  const long long ctas = (items + ITEMS - 1) / ITEMS;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kBoundThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, bound_blocks_kernel<FMT, HD, WPI>, a);
}

// A block's rows of one head up to 8 KB go to one warp (at most 16 loads a
// lane); larger ones to the whole CTA's 8.
template <int FMT, int HD>
cudaError_t launch_hd(const BoundArgs& a, cudaStream_t s) {
  constexpr int ROWB = HD * (FMT == KVQ_F16 ? 2 : 1);
  if ((ROWB << a.pool.bs_log2) <= 8192) return launch_wpi<FMT, HD, 1>(a, s);
  return launch_wpi<FMT, HD, kBoundThreads / 32>(a, s);
}

}  // namespace

cudaError_t launch_bound_blocks(int fmt, int hd, const BoundArgs& a, cudaStream_t s) {
  if (fmt == KVQ_F16) {
    if (hd == 64) return launch_hd<KVQ_F16, 64>(a, s);
    if (hd == 128) return launch_hd<KVQ_F16, 128>(a, s);
    return launch_hd<KVQ_F16, 256>(a, s);
  }
  if (hd == 64) return launch_hd<KVQ_Q8, 64>(a, s);
  if (hd == 128) return launch_hd<KVQ_Q8, 128>(a, s);
  return launch_hd<KVQ_Q8, 256>(a, s);
}

}  // namespace kvq
