// kvq_rotary.cu -- norms of each head's query and key, rotary positions, and
// the append of the new keys and values, in one pass (kvq_append_rotary).
//
//   x' = x * rsqrt(mean(x^2) + eps) * w              (q and k, where w is given)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t)  t = position * inv_freq
//
// The pass reads q, k and v once and writes q (fp32) and the cache rows: HBM
// bounds it.  A warp takes one token and every parts-th block of 32 / LPR
// heads; LPR = HD / 8 lanes hold a head, 8 consecutive dims each, so the
// angles of a lane's dims are the same for all heads of the token: their
// sines and cosines are taken once and stay in registers, and a pair's other
// half is a lane's own (interleaved) or one shuffle away.  The quantisers
// are the appends' own, so the cache bytes are kvq_append's of the same fp32
// rows.
#include <cuda_bf16.h>

#include "kvq_quant.cuh"

namespace kvq {
namespace {

constexpr int kRotWarps = 4;
constexpr int VPL = 8;

template <int T>
struct Elem;
template <>
struct Elem<KVQ_T_F32> {
  using type = float;
  static constexpr int kVecs = 2;
};
template <>
struct Elem<KVQ_T_F16> {
  using type = __half;
  static constexpr int kVecs = 1;
};
template <>
struct Elem<KVQ_T_BF16> {
  using type = __nv_bfloat16;
  static constexpr int kVecs = 1;
};

// 8 consecutive values as they lie in memory (read once: not kept in L1)
template <int T>
struct Raw {
  uint4 w[Elem<T>::kVecs];
};

template <int T>
__device__ __forceinline__ Raw<T> load8(const void* base, long long at, bool live) {
  Raw<T> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const typename Elem<T>::type*>(base) + at);
#pragma unroll
  for (int i = 0; i < Elem<T>::kVecs; ++i) r.w[i] = live ? __ldcs(p + i) : make_uint4(0, 0, 0, 0);
  return r;
}

template <int T>
__device__ __forceinline__ void widen8(const Raw<T>& r, float (&x)[VPL]) {
#pragma unroll
  for (int i = 0; i < Elem<T>::kVecs; ++i) {
    const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (T == KVQ_T_F32) {
        x[4 * i + e] = __uint_as_float(w[e]);
      } else if constexpr (T == KVQ_T_F16) {
        x[2 * e] = half_lo(w[e]);
        x[2 * e + 1] = half_hi(w[e]);
      } else {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  }
}

// Sine and cosine of pos * f.  The angle in half turns is t = pos * f / pi;
// its even part is taken off before the functions see it.  Angles up to 2^22
// are held as an fp32 pair (a position up to 2^24 is exact, p + e = pos * f
// exactly, and 1 / pi is a pair too: t is off by about 2^-46 of itself);
// larger ones take fp64, which the SM runs at a sixty-fourth of the rate.
__device__ __forceinline__ void turn(int pos, float f, float& c, float& s) {
  constexpr double kInvPi = 0.31830988618379067154;
  float r;
  const float x = (float)pos, p = x * f;
  if (abs(pos) <= (1 << 24) && fabsf(p) < 4194304.0f) {
    constexpr float hi = (float)kInvPi, lo = (float)(kInvPi - (double)hi);
    const float e = fmaf(x, f, -p);
    const float t = p * hi, d = fmaf(p, hi, -t) + fmaf(p, lo, e * hi);
    r = (t - 2.0f * rintf(0.5f * t)) + d;
  } else {
    const double t = (double)pos * (double)f * kInvPi;
    r = (float)(t - 2.0 * rint(0.5 * t));
  }
  sincospif(r, &s, &c);
}

template <int FMT, int HD, int T>
__global__ void __launch_bounds__(kRotWarps * 32) append_rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int LPR = HD / VPL;   // lanes of a head
  constexpr int RPW = 32 / LPR;   // heads a warp holds
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, j = lane & (LPR - 1), sub = lane / LPR;
  const unsigned wid = blockIdx.x * kRotWarps + (threadIdx.x >> 5);
  const int tok = (int)fdiv(wid, a.div_parts), part = (int)wid - tok * a.parts;
  if (tok >= a.n_tok) return;   // warp-uniform
  const int n_kv = a.pool.n_kv;
  const int qb = (a.n_q + RPW - 1) / RPW, kb = (n_kv + RPW - 1) / RPW, nb = qb + 2 * kb;

  // the heads of block b: 0 .. qb - 1 queries, then keys, then values
  auto fetch = [&](int b) -> Raw<T> {
    const bool is_q = b < qb, is_k = !is_q && b < qb + kb;
    const int h = (is_q ? b : is_k ? b - qb : b - qb - kb) * RPW + sub;
    const void* base = is_q ? a.q : is_k ? a.k : a.v;
    const long long stride = is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride;
    return load8<T>(base, tok * stride + h * HD + j * VPL, b < nb && h < (is_q ? a.n_q : n_kv));
  };
  Raw<T> next = fetch(part);

  const int seq = __ldg(a.tok_seq + tok), pos = __ldg(a.tok_pos + tok);
  if (seq < 0 || seq >= a.n_seq || pos < 0) return;   // padding
  // the token's cell: row of KV head 0, -1 if it has none
  long long row0 = -1;
  const int bs = 1 << a.pool.bs_log2;
  if ((pos >> a.pool.bs_log2) < a.max_blocks) {
    const int blk = __ldg(a.block_table + (size_t)seq * a.max_blocks + (pos >> a.pool.bs_log2));
    if (blk >= 0 && blk < a.pool.n_blocks) row0 = (long long)blk * n_kv * bs + (pos & (bs - 1));
  }

  // cosines and signed sines of this lane's dims (a multiple of 16 dims
  // rotate, so a lane's 8 do or do not, and its partner is one lane)
  const int d0 = j * VPL, half = a.rot_dim / 2;
  const bool rot = d0 < a.rot_dim, upper = !a.interleaved && d0 >= half;
  float cs[VPL], sn[VPL];
  int partner = lane;
  if (rot && part < qb + kb) {
    const int i0 = a.interleaved ? d0 / 2 : upper ? d0 - half : d0;
    if (!a.interleaved) partner = upper ? lane - half / VPL : lane + half / VPL;
#pragma unroll
    for (int e = 0; e < VPL; ++e) {
      if (a.interleaved && e >= VPL / 2) break;
      const int i = i0 + e;
      int p = pos;
      if (a.positions != nullptr) {
        const int ax = a.pair_axis != nullptr ? min(max(__ldg(a.pair_axis + i), 0), a.n_axes - 1) : 0;
        p = __ldg(a.positions + (size_t)ax * a.n_tok + tok);
      }
      float c, s;
      turn(p, __ldg(a.inv_freq + i), c, s);
      cs[e] = c * a.gain;
      sn[e] = (upper || a.interleaved ? s : -s) * a.gain;
    }
  }

  for (int b = part; b < nb; b += a.parts) {
    float x[VPL];
    widen8<T>(next, x);
    next = fetch(b + a.parts);
    const bool is_q = b < qb, is_v = b >= qb + kb;
    const int h = (is_q ? b : is_v ? b - qb - kb : b - qb) * RPW + sub;
    const bool live = h < (is_q ? a.n_q : n_kv);
    if (!is_v) {
      const float* w = is_q ? a.q_norm : a.k_norm;
      if (w != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < VPL; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float rs = rsqrtf(ss * (1.0f / HD) + a.eps);
        const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + d0)),
                     w1 = __ldg(reinterpret_cast<const float4*>(w + d0 + 4));
        const float ww[VPL] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int e = 0; e < VPL; ++e) x[e] *= rs * ww[e];
      }
      if (a.interleaved) {
        if (rot) {
#pragma unroll
          for (int e = 0; e < VPL; e += 2) {
            const float c = cs[e / 2], s = sn[e / 2], u = x[e], v = x[e + 1];
            x[e] = fmaf(u, c, -(v * s));
            x[e + 1] = fmaf(v, c, u * s);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < VPL; ++e) {
          const float y = __shfl_sync(0xffffffffu, x[e], partner);
          if (rot) x[e] = fmaf(x[e], cs[e], y * sn[e]);
        }
      }
    }
    if (is_q) {
      if (live) {
        float4* dst = reinterpret_cast<float4*>(a.q_out + ((size_t)tok * a.n_q + h) * HD + d0);
        dst[0] = make_float4(x[0], x[1], x[2], x[3]);
        dst[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
      continue;
    }
    const long long dr = live && row0 >= 0 ? row0 + (long long)h * bs : -1;
    if constexpr (FMT == KVQ_F16) {
      if (dr >= 0)
        *reinterpret_cast<uint4*>(static_cast<__half*>(is_v ? a.v_dst : a.k_dst) + dr * HD + d0) =
            make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]),
                       pack_half2(x[6], x[7]));
    } else if (FMT == KVQ_K8V4 && is_v) {
      wht_group<VPL, LPR>(x, lane);
      q4_lanes<HD, VPL>(x, dr, j, lane, static_cast<uint8_t*>(a.v_dst), a.vs_dst);
    } else {
      q8_lanes<HD, VPL, LPR>(x, dr, j, static_cast<int8_t*>(is_v ? a.v_dst : a.k_dst),
                             is_v ? a.vs_dst : a.ks_dst);
    }
  }
}

template <int FMT, int HD, int T>
cudaError_t launch(RotaryArgs a, int sms, cudaStream_t s) {
  constexpr int RPW = 32 / (HD / VPL);
  const int nb = (a.n_q + RPW - 1) / RPW + 2 * ((a.pool.n_kv + RPW - 1) / RPW);
  // enough warps to fill the SMs, down to one head block a warp
  const long long want = (long long)sms * 32;
  long long parts = (want + a.n_tok - 1) / a.n_tok;
  a.parts = (int)(parts < 1 ? 1 : parts > nb ? nb : parts);
  a.div_parts = make_fastdiv((unsigned)a.parts);
  const long long warps = (long long)a.n_tok * a.parts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + kRotWarps - 1) / kRotWarps));
  cfg.blockDim = dim3(kRotWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_rotary_kernel<FMT, HD, T>, a);
}

template <int FMT, int HD>
cudaError_t launch_type(int type, const RotaryArgs& a, int sms, cudaStream_t s) {
  switch (type) {
    case KVQ_T_F32: return launch<FMT, HD, KVQ_T_F32>(a, sms, s);
    case KVQ_T_F16: return launch<FMT, HD, KVQ_T_F16>(a, sms, s);
    case KVQ_T_BF16: return launch<FMT, HD, KVQ_T_BF16>(a, sms, s);
    default: return cudaErrorInvalidValue;
  }
}

template <int HD>
cudaError_t launch_fmt(int fmt, int type, const RotaryArgs& a, int sms, cudaStream_t s) {
  switch (fmt) {
    case KVQ_F16: return launch_type<KVQ_F16, HD>(type, a, sms, s);
    case KVQ_Q8: return launch_type<KVQ_Q8, HD>(type, a, sms, s);
    case KVQ_K8V4: return launch_type<KVQ_K8V4, HD>(type, a, sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_append_rotary(int fmt, int hd, int type, RotaryArgs a, int sms, cudaStream_t s) {
  switch (hd) {
    case 64: return launch_fmt<64>(fmt, type, a, sms, s);
    case 128: return launch_fmt<128>(fmt, type, a, sms, s);
    case 256: return launch_fmt<256>(fmt, type, a, sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
