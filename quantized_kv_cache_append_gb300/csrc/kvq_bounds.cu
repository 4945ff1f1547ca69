// kvq_bounds.cu -- bounds of each cache block's keys (kvq_bound_blocks).
//
// For a block's live cells and one KV head, lo[d] = min and hi[d] = max over
// the cells of the dequantised key K[c][d]; per 64 dims, s = 2^e with the
// smallest e in [-24, 16] that gives 127 s >= max(|lo|, |hi|), and the codes
// floor(lo / s) and ceil(hi / s).  All of it is exact: the dequantised keys
// are fp16 values or products of an int8 code and an fp16 scale, which fp32
// holds exactly, and a division by a power of two does not round.
//
// A work item is one (block, KV head): block_size contiguous rows of K.  One
// warp or the CTA's 8 read it with 16-byte (int8: 8-byte) loads, each lane
// always at the same 8 dims, the running minima and maxima in registers.  The lanes of the
// same dims meet by a halving exchange (each step a lane keeps half of its
// dims), which leaves HD / 32 consecutive dims a lane; 8 warps meet through
// shared memory.  CTAs are persistent and fetch the next item's block id
// before the current item's rows.  FP16 rows stay fp16 pairs throughout.
// int8 codes become fp32 values in one byte permute and half a packed FMA:
// the bytes 0x47 00 uu 00 are the float 32768 + u, and (32768 + u) s - 32896 s
// is (u - 128) s exactly (32896 s has at most 20 significant bits); two rows
// share a three-input minimum and maximum.  The rows are read with ordinary
// loads: the attention that follows reads the newest blocks again, from L2
// (streaming loads gain 2 % on a whole prompt and lose 2 us on a step).
//
// Bound by the read of K.  One GB300: 262144 FP16 cells x 2 heads x 256 dims
// (268 MB) 44 us, 6.1 TB/s, 90 % of the measured copy rate; the newest block
// of 16 sequences (8 heads x 128 dims, blocks of 256) 3.4 us, a launch with
// one dependent chain of loads.  131072 int8 cells x 8 heads x 128 dims in
// blocks of 64 37 us, 3.8 TB/s: 4.2 instructions a code keep the ALU half
// busy and the loads' latency shows between them (16-byte loads with two
// CTAs an SM, batches fetched ahead and 2 to 5 CTAs an SM all took 35-45 us).
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "kvq_internal.cuh"
#include "kvq_ptx.cuh"

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

__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// (x0, x1) s + t, packed
__device__ __forceinline__ float2 fma2(uint32_t x0, uint32_t x1, float s, float t) {
  float2 d;
  asm("{\n .reg .b64 x, s, t, d;\n mov.b64 x, {%2, %3};\n mov.b64 s, {%4, %4};\n mov.b64 t, {%5, %5};\n"
      " fma.rn.f32x2 d, x, s, t;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "r"(x0), "r"(x1), "f"(s), "f"(t));
  return d;
}
// 4 int8 codes times s
__device__ __forceinline__ void widen4(uint32_t w, float s, float t, float (&x)[4]) {
  w ^= 0x80808080u;
  const float2 a = fma2(prmt(w, 0x47000000u, 0x7404u), prmt(w, 0x47000000u, 0x7414u), s, t);
  const float2 b = fma2(prmt(w, 0x47000000u, 0x7424u), prmt(w, 0x47000000u, 0x7434u), s, t);
  x[0] = a.x;
  x[1] = a.y;
  x[2] = b.x;
  x[3] = b.y;
}

__device__ __forceinline__ float lower(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ float upper(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ __half2 lower(__half2 a, __half2 b) { return __hmin2(a, b); }
__device__ __forceinline__ __half2 upper(__half2 a, __half2 b) { return __hmax2(a, b); }

// x[N] of lanes l and l ^ OFF, l ^ (OFF / 2), .. l ^ LAST combined, each step
// keeping the half of x that the lane's bit names: N LAST / (2 OFF) values are
// left in x[0 ..].
template <bool MAX, int N, int OFF, int LAST, class T>
__device__ __forceinline__ void halve(T* x, int lane) {
  if constexpr (OFF >= LAST) {
    const bool up = lane & OFF;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const T keep = up ? x[i + N / 2] : x[i], give = up ? x[i] : x[i + N / 2];
      const T got = __shfl_xor_sync(kAll, give, OFF);
      x[i] = MAX ? upper(keep, got) : lower(keep, got);
    }
    halve<MAX, N / 2, OFF / 2, LAST>(x, lane);
  }
}

// FMT: KVQ_F16, or KVQ_Q8 for both int8-K formats.  WPI warps per item.
template <int FMT, int HD, int WPI>
__global__ void __launch_bounds__(kBoundThreads, FMT == KVQ_F16 ? 5 : 3)
    bound_blocks_kernel(BoundArgs a) {
  constexpr bool I8 = FMT != KVQ_F16;
  constexpr int VD = 8;                   // dims per load (16 or 8 bytes)
  constexpr int LPR = HD / VD;            // lanes per row
  constexpr int RPW = 32 / LPR;           // rows a warp reads at once
  constexpr int NG = HD / kGroup;
  constexpr int ITEMS = kBoundThreads / 32 / WPI;   // items per CTA
  constexpr int LG = kGroup / VD;         // lanes of one 64-dim group in a row
  constexpr int S = HD / 32;              // dims a lane ends with
  constexpr int STEP = RPW * WPI;         // rows an item's warps read at once
  static_assert(WPI == 1 || ITEMS == 1, "an item is one warp's or the CTA's");
  __shared__ __align__(16) float s_red[WPI > 1 ? 2 : 1][WPI > 1 ? WPI : 1][2][WPI > 1 ? HD : 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wi = WPI > 1 ? warp : 0;
  const int l = lane % LPR, rg = lane / LPR, r0 = wi * RPW + rg;
  const int bs_log2 = a.pool.bs_log2;
  const uint32_t items = (uint32_t)a.n_seq * (uint32_t)a.touched * (uint32_t)a.pool.n_kv;

  // item = (sequence, touched block, KV head), heads innermost: its block (-1:
  // nothing to do), live cells and head
  struct Item {
    int blk, live, h;
  };
  auto find = [&](uint32_t item) -> Item {
    Item x = {-1, 0, 0};
    if (item >= items) return x;
    const uint32_t sb = fdiv(item, a.div_nkv);
    x.h = (int)(item - sb * (uint32_t)a.pool.n_kv);
    const uint32_t b = fdiv(sb, a.div_touched);
    const long long cap = (long long)a.max_blocks << bs_log2;
    const long long len = min((long long)__ldg(a.ctx_lens + b), cap);
    const int start = a.ctx_start != nullptr ? max(__ldg(a.ctx_start + b), 0) : 0;
    const long long j = (start >> bs_log2) + (int)(sb - b * (uint32_t)a.touched);
    if (start < len && (j << bs_log2) < len) {
      const int blk = __ldg(a.block_table + (size_t)b * a.max_blocks + j);
      x.blk = blk >= 0 && blk < a.pool.n_blocks ? blk : -1;
      x.live = (int)min(1LL << bs_log2, len - (j << bs_log2));
    }
    return x;
  };

  uint32_t item = blockIdx.x * ITEMS + (WPI > 1 ? 0 : warp);
  Item next = find(item);
  int buf = 0;
  for (; item < items; item += gridDim.x * ITEMS) {
    const Item it = next;
    next = find(item + gridDim.x * ITEMS);
    if (it.blk < 0) continue;             // (uniform over the item's warps)
    const size_t row0 = ((size_t)it.blk * a.pool.n_kv + it.h) << bs_log2;
    float lo[S], hi[S];
    if constexpr (!I8) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __half*>(a.pool.k) + row0 * HD) + l;
      __half2 mn[4], mx[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        mn[e] = __halves2half2(__ushort_as_half(0x7c00), __ushort_as_half(0x7c00));
        mx[e] = __halves2half2(__ushort_as_half(0xfc00), __ushort_as_half(0xfc00));
      }
#pragma unroll 4
      for (int r = r0; r < it.live; r += STEP) {
        const uint4 u = __ldg(src + (size_t)r * LPR);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 x = *reinterpret_cast<const __half2*>(&w[e]);
          mn[e] = __hmin2(mn[e], x);   // (a NaN operand is passed over)
          mx[e] = __hmax2(mx[e], x);
        }
      }
      halve<false, 4, 16, LPR>(mn, lane);
      halve<true, 4, 16, LPR>(mx, lane);
#pragma unroll
      for (int e = 0; e < S / 2; ++e) {
        lo[2 * e] = __low2float(mn[e]);
        lo[2 * e + 1] = __high2float(mn[e]);
        hi[2 * e] = __low2float(mx[e]);
        hi[2 * e + 1] = __high2float(mx[e]);
      }
    } else {
      const uint2* src = reinterpret_cast<const uint2*>(static_cast<const int8_t*>(a.pool.k) + row0 * HD) + l;
      const __half* sc = a.pool.ks + row0 * NG + l / LG;
      float mn[VD], mx[VD];
#pragma unroll
      for (int e = 0; e < VD; ++e) {
        mn[e] = INFINITY;
        mx[e] = -INFINITY;
      }
#pragma unroll 4
      for (int r = r0; r < it.live; r += 2 * STEP) {
        const int r2 = r + STEP < it.live ? r + STEP : r;
        const uint2 u = __ldg(src + (size_t)r * LPR), v = __ldg(src + (size_t)r2 * LPR);
        const float su = __half2float(__ldg(sc + (size_t)r * NG)), sv = __half2float(__ldg(sc + (size_t)r2 * NG));
        const float tu = -32896.0f * su, tv = -32896.0f * sv;
        const uint32_t wu[2] = {u.x, u.y}, wv[2] = {v.x, v.y};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x[4], y[4];
          widen4(wu[e], su, tu, x);
          widen4(wv[e], sv, tv, y);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            mn[4 * e + k] = min3(mn[4 * e + k], x[k], y[k]);
            mx[4 * e + k] = max3(mx[4 * e + k], x[k], y[k]);
          }
        }
      }
      halve<false, VD, 16, LPR>(mn, lane);
      halve<true, VD, 16, LPR>(mx, lane);
#pragma unroll
      for (int e = 0; e < S; ++e) {
        lo[e] = mn[e];
        hi[e] = mx[e];
      }
    }
    const int d0 = l * VD + rg * S;       // the lane's dims
    if constexpr (WPI > 1) {
#pragma unroll
      for (int e = 0; e < S; e += 2) {
        *reinterpret_cast<float2*>(&s_red[buf][wi][0][d0 + e]) = make_float2(lo[e], lo[e + 1]);
        *reinterpret_cast<float2*>(&s_red[buf][wi][1][d0 + e]) = make_float2(hi[e], hi[e + 1]);
      }
      __syncthreads();
      // one warp finishes while the others start the next item's rows in the
      // other buffer
      const int use = buf;
      buf ^= 1;
      if (wi != 0) continue;
#pragma unroll
      for (int w = 1; w < WPI; ++w)
#pragma unroll
        for (int e = 0; e < S; e += 2) {
          const float2 x = *reinterpret_cast<const float2*>(&s_red[use][w][0][d0 + e]);
          const float2 y = *reinterpret_cast<const float2*>(&s_red[use][w][1][d0 + e]);
          lo[e] = fminf(lo[e], x.x);
          lo[e + 1] = fminf(lo[e + 1], x.y);
          hi[e] = fmaxf(hi[e], y.x);
          hi[e + 1] = fmaxf(hi[e + 1], y.y);
        }
    }
    // scale of the 64 dims this lane's belong to (a dim without any number: 0)
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < S; ++e) {
      if (lo[e] > hi[e]) lo[e] = hi[e] = 0.f;
      m = fmaxf(m, fmaxf(fabsf(lo[e]), fabsf(hi[e])));
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
      if (off < LG || off >= LPR) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
    const int e2 = scale_exponent(m, -24, 16);
    const float inv = pow2f_exact(-e2);
    uint32_t cl[(S + 3) / 4], ch[(S + 3) / 4];
#pragma unroll
    for (int i = 0; i < (S + 3) / 4; ++i) cl[i] = ch[i] = 0;
#pragma unroll
    for (int e = 0; e < S; ++e) {
      const int x = (int)fminf(fmaxf(floorf(lo[e] * inv), -127.f), 127.f);
      const int y = (int)fminf(fmaxf(ceilf(hi[e] * inv), -127.f), 127.f);
      cl[e / 4] |= (uint32_t)(x & 0xff) << (8 * (e % 4));
      ch[e / 4] |= (uint32_t)(y & 0xff) << (8 * (e % 4));
    }
    int8_t* dst = a.bounds + ((size_t)it.blk * a.pool.n_kv + it.h) * 2 * HD + d0;
    if constexpr (S == 2) {
      *reinterpret_cast<uint16_t*>(dst) = (uint16_t)cl[0];
      *reinterpret_cast<uint16_t*>(dst + HD) = (uint16_t)ch[0];
    } else if constexpr (S == 4) {
      *reinterpret_cast<uint32_t*>(dst) = cl[0];
      *reinterpret_cast<uint32_t*>(dst + HD) = ch[0];
    } else {
      *reinterpret_cast<uint2*>(dst) = make_uint2(cl[0], cl[S > 4 ? 1 : 0]);
      *reinterpret_cast<uint2*>(dst + HD) = make_uint2(ch[0], ch[S > 4 ? 1 : 0]);
    }
    if (l % LG == 0 && rg == 0)
      a.scales[((size_t)it.blk * a.pool.n_kv + it.h) * NG + l / LG] = pow2f_exact(e2);
  }
}

template <int FMT, int HD, int WPI>
cudaError_t launch_wpi(const BoundArgs& a, int sms, cudaStream_t s) {
  constexpr int ITEMS = kBoundThreads / 32 / WPI;
  static ContextCache<int> cache;
  int per_sm = 0;
  if (!per_context(cache, &per_sm, [](int* v) {
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, bound_blocks_kernel<FMT, HD, WPI>, kBoundThreads,
                                                             0) == cudaSuccess &&
               *v > 0;
      }))
    return cudaErrorInvalidConfiguration;
  const long long items = (long long)a.n_seq * a.touched * a.pool.n_kv;
  long long ctas = (items + ITEMS - 1) / ITEMS;
  if (ctas > (long long)per_sm * sms) ctas = (long long)per_sm * sms;
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
// lane), larger ones to the CTA's 8, and so do smaller ones when there are
// too few to give every SM 8 warps.
template <int FMT, int HD>
cudaError_t launch_hd(const BoundArgs& a, int sms, cudaStream_t s) {
  constexpr int ROWB = HD * (FMT == KVQ_F16 ? 2 : 1);
  const long long items = (long long)a.n_seq * a.touched * a.pool.n_kv;
  if ((ROWB << a.pool.bs_log2) <= 8192 && items >= 8LL * sms) return launch_wpi<FMT, HD, 1>(a, sms, s);
  return launch_wpi<FMT, HD, kBoundThreads / 32>(a, sms, s);
}

}  // namespace

cudaError_t launch_bound_blocks(int fmt, int hd, const BoundArgs& a, int sms, cudaStream_t s) {
  if (fmt == KVQ_F16) {
    if (hd == 64) return launch_hd<KVQ_F16, 64>(a, sms, s);
    if (hd == 128) return launch_hd<KVQ_F16, 128>(a, sms, s);
    return launch_hd<KVQ_F16, 256>(a, sms, s);
  }
  if (hd == 64) return launch_hd<KVQ_Q8, 64>(a, sms, s);
  if (hd == 128) return launch_hd<KVQ_Q8, 128>(a, sms, s);
  return launch_hd<KVQ_Q8, 256>(a, sms, s);
}

}  // namespace kvq
