// kvq_rotary.cu -- norms of each head's query and key, rotary positions, and
// the append of the new keys and values, in one pass (kvq_append_rotary).
//
//   x' = x * rsqrt(mean(x^2) + eps) * w              (q and k, where w is given)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t)  t = position * inv_freq
//
// The pass reads q, k and v once and writes q (fp32) and the cache rows: HBM
// bounds it, if the instructions stay few.  A CTA takes one token (for few
// tokens, a part of its heads): its threads take the sines and cosines of the
// token's pairs once, into shared memory.  LPR = HD / 8 lanes of a warp hold a
// head, 8 consecutive dims each, and keep what those dims of every head are
// multiplied with in registers, the norm's weights included:
//
//   out = rs * (x * (w cos) + y * (w' sin))     y the pair's other value, w'
//                                               its weight, rs the head's norm
//
// y is a lane's own value (interleaved) or one shuffle of the raw words away.
// The quantisers are the appends' own, so the cache bytes are kvq_append's of
// the same fp32 rows.
#include <cuda_bf16.h>

#include "kvq_quant.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace {

constexpr int kRotWarps = 2;
// CTAs an SM that few tokens are spread over, half of what is resident: 512 tokens
// of 32/8 heads 5.25 us, 256 4.0 (4: 6.9 and 4.5, 14: 6.1 and 5.2, 20: 7.7 and 5.9).
constexpr int kRotCtas = 7;
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
__device__ __forceinline__ Raw<T> load8(const typename Elem<T>::type* base, int at, bool live) {
  Raw<T> r;
  const uint4* p = reinterpret_cast<const uint4*>(base + at);
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

__device__ __forceinline__ void load_floats(const float* p, float (&x)[VPL]) {   // 16-byte aligned
  const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 4);
  x[0] = u.x;
  x[1] = u.y;
  x[2] = u.z;
  x[3] = u.w;
  x[4] = v.x;
  x[5] = v.y;
  x[6] = v.z;
  x[7] = v.w;
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

// 28 warps an SM and 2 blocks of queries in flight a warp: 4096 bf16 tokens of
// 32 + 2 x 8 heads of 128 dims 25.6 us (4.9 TB/s; 16384 tokens 5.6 TB/s), 16381
// fp32 tokens of 16 + 2 x 2 heads of 256 dims with 3 axes 95 us (97 % of the copy
// rate).  CTAs of 1 warp 33 and 106 us, of 4 warps 32 and 109; 20 warps an SM 28.5
// and 100, 32 27.5 and 110.  A first form with 12 blocks a warp, each warp taking
// its own sines, ran 235 instructions a block and 29.3 and 106 us.
template <int FMT, int HD, int T>
__global__ void __launch_bounds__(kRotWarps * 32, 14) append_rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int LPR = HD / VPL;   // lanes of a head
  constexpr int RPW = 32 / LPR;   // heads a warp holds
  constexpr int UQ = 2, UK = 1;   // blocks of queries, of keys and of values in flight
  using E = typename Elem<T>::type;
  __shared__ __align__(16) float s_cos[HD / 2], s_sin[HD / 2];   // of each pair, times the gain
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, j = lane & (LPR - 1), sub = lane / LPR;
  const int tok = blockIdx.x, n_kv = a.pool.n_kv, bs = 1 << a.pool.bs_log2;
  // blocks of RPW heads: 0 .. qb - 1 queries, then keys, then values; this warp
  // takes every n_parts-th: bq, bk and bv the first of each kind.  Their
  // values are on the way before the token's place is known.
  const int n_parts = gridDim.y * kRotWarps;
  const int bq = blockIdx.y * kRotWarps + (threadIdx.x >> 5);
  auto from = [&](int mod) -> int { return bq >= mod ? bq - mod : bq - mod + n_parts; };   // (bq - mod) mod n_parts
  const int bk = from(a.mod_k), bv = from(a.mod_v);   // counted within their kind
  // (h < n leaves out the blocks behind the last too)
  auto at = [&](const void* rows, long long stride, int b) -> const E* {
    return static_cast<const E*>(rows) + (tok * stride + (b * RPW + sub) * HD + j * VPL);
  };
  const int step = n_parts * RPW;   // heads from block to block
  Raw<T> rq[UQ], rk[UK], rv[UK];
  {
    const E *pq = at(a.q, a.q_stride, bq), *pk = at(a.k, a.k_stride, bk), *pv = at(a.v, a.v_stride, bv);
    const int hq = bq * RPW + sub, hk = bk * RPW + sub, hv = bv * RPW + sub;
#pragma unroll
    for (int u = 0; u < UQ; ++u) rq[u] = load8<T>(pq, u * step * HD, hq + u * step < a.n_q);
#pragma unroll
    for (int u = 0; u < UK; ++u) {
      rk[u] = load8<T>(pk, u * step * HD, hk + u * step < n_kv);
      rv[u] = load8<T>(pv, u * step * HD, hv + u * step < n_kv);
    }
  }
  const int seq = __ldg(a.tok_seq + tok), pos = __ldg(a.tok_pos + tok);
  if (seq < 0 || seq >= a.n_seq || pos < 0) return;   // padding (the whole CTA)
  for (int i = threadIdx.x; i < a.rot_dim / 2; i += kRotWarps * 32) {
    int p = pos;
    if (a.positions != nullptr) {
      const int ax = a.pair_axis != nullptr ? min(max(__ldg(a.pair_axis + i), 0), a.n_axes - 1) : 0;
      p = __ldg(a.positions + (size_t)ax * a.n_tok + tok);
    }
    float c, s;
    turn(p, __ldg(a.inv_freq + i), c, s);
    s_cos[i] = c * a.gain;
    s_sin[i] = s * a.gain;
  }
  // the token's cell: row of KV head 0, -1 if it has none
  long long row0 = -1;
  if ((pos >> a.pool.bs_log2) < a.max_blocks) {
    const int blk = __ldg(a.block_table + (size_t)seq * a.max_blocks + (pos >> a.pool.bs_log2));
    if (blk >= 0 && blk < a.pool.n_blocks) row0 = (long long)blk * n_kv * bs + (pos & (bs - 1));
  }
  __syncthreads();

  // cosines and signed sines of this lane's dims (a multiple of 16 dims
  // rotate, so a lane's 8 do or do not, and its partner is one lane)
  const int d0 = j * VPL, half = a.rot_dim / 2;
  const bool inter = a.interleaved != 0, rot = d0 < a.rot_dim, upper = !inter && d0 >= half;
  const int partner = inter || !rot ? lane : upper ? lane - half / VPL : lane + half / VPL;
  const int p0 = inter || !rot ? d0 : upper ? d0 - half : d0 + half;   // its first dim
  auto turns = [&](float (&cs)[VPL], float (&sn)[VPL]) {
    if (!rot) {
#pragma unroll
      for (int e = 0; e < VPL; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
      }
    } else if (inter) {
      const float4 c = *reinterpret_cast<const float4*>(s_cos + d0 / 2), t = *reinterpret_cast<const float4*>(s_sin + d0 / 2);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int e = 0; e < VPL; ++e) {
        cs[e] = cc[e / 2];
        sn[e] = e & 1 ? ss[e / 2] : -ss[e / 2];
      }
    } else {
      const int i = upper ? p0 : d0;
      load_floats(s_cos + i, cs);
      load_floats(s_sin + i, sn);
      if (!upper) {
#pragma unroll
        for (int e = 0; e < VPL; ++e) sn[e] = -sn[e];
      }
    }
  };

  // one kind of heads: this warp's blocks of them from b on, the first in r; n heads
  auto heads = [&](auto& r, const void* rows, long long stride, int b, int n, const float* w, bool turned, auto put) {
    constexpr int U = sizeof(r) / sizeof(Raw<T>);
    if (b * RPW >= n) return;
    float cw[VPL], sw[VPL];
    const bool norm = w != nullptr;
    if (turned) {
      turns(cw, sw);
      if (norm) {
        float wd[VPL], wp[VPL];
        load_floats(w + d0, wd);
        load_floats(w + p0, wp);
#pragma unroll
        for (int e = 0; e < VPL; ++e) {
          cw[e] *= wd[e];
          sw[e] *= inter ? wp[e ^ 1] : wp[e];
        }
      }
    }
    while (true) {
      // 16-bit types: the next blocks are on the way while these are worked on (4096
      // bf16 tokens 28.4 -> 25.6 us; fp32 has no registers for it, 34 -> 42)
      constexpr bool kAhead = T != KVQ_T_F32;
      Raw<T> next[U];
      auto fetch = [&](int b1) {
        const E* p = at(rows, stride, b1);
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = load8<T>(p, u * step * HD, b1 * RPW + sub + u * step < n);
      };
      if constexpr (kAhead) fetch(b + U * n_parts);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (b * RPW >= n) break;   // warp-uniform
        const int h = b * RPW + sub;
        float x[VPL];
        widen8<T>(r[u], x);
        if (turned) {
          float rs = 1.f;
          if (norm) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int e = 0; e < VPL; e += 2) fma_f32x2(s0, s1, x[e], x[e + 1], x[e], x[e + 1], s0, s1);
            float ss = s0 + s1;
#pragma unroll
            for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            rs = rsqrtf(ss * (1.0f / HD) + a.eps);
          }
          float y[VPL];
          if (inter) {
#pragma unroll
            for (int e = 0; e < VPL; ++e) y[e] = rot ? x[e ^ 1] : 0.f;   // (not 0 * infinity)
          } else {
            Raw<T> o;
#pragma unroll
            for (int i = 0; i < Elem<T>::kVecs; ++i) {
              o.w[i].x = __shfl_sync(0xffffffffu, r[u].w[i].x, partner);
              o.w[i].y = __shfl_sync(0xffffffffu, r[u].w[i].y, partner);
              o.w[i].z = __shfl_sync(0xffffffffu, r[u].w[i].z, partner);
              o.w[i].w = __shfl_sync(0xffffffffu, r[u].w[i].w, partner);
              if (!rot) o.w[i] = make_uint4(0, 0, 0, 0);
            }
            widen8<T>(o, y);
          }
#pragma unroll
          for (int e = 0; e < VPL; e += 2) {
            mul_f32x2(x[e], x[e + 1], x[e], x[e + 1], cw[e], cw[e + 1]);
            fma_f32x2(x[e], x[e + 1], y[e], y[e + 1], sw[e], sw[e + 1], x[e], x[e + 1]);
            if (norm) mul_f32x2(x[e], x[e + 1], x[e], x[e + 1], rs, rs);
          }
        }
        put(x, h, h < n);
        b += n_parts;
      }
      if (b * RPW >= n) return;
      if constexpr (!kAhead) fetch(b);
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = next[u];
    }
  };

  float* q_out = a.q_out + (size_t)tok * a.n_q * HD + d0;
  heads(rq, a.q, a.q_stride, bq, a.n_q, a.q_norm, true, [&](const float (&x)[VPL], int h, bool live) {
    if (live) {
      float4* dst = reinterpret_cast<float4*>(q_out + h * HD);
      dst[0] = make_float4(x[0], x[1], x[2], x[3]);
      dst[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  });
  auto cache_row = [&](int h, bool live) -> long long { return live && row0 >= 0 ? row0 + (long long)h * bs : -1; };
  auto put16 = [&](void* dst, const float (&x)[VPL], long long dr) {
    if (dr >= 0)
      *reinterpret_cast<uint4*>(static_cast<__half*>(dst) + dr * HD + d0) =
          make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
  };
  heads(rk, a.k, a.k_stride, bk, n_kv, a.k_norm, true, [&](const float (&x)[VPL], int h, bool live) {
    const long long dr = cache_row(h, live);
    if constexpr (FMT == KVQ_F16) put16(a.k_dst, x, dr);
    else q8_lanes<HD, VPL, LPR>(x, dr, j, static_cast<int8_t*>(a.k_dst), a.ks_dst);
  });
  heads(rv, a.v, a.v_stride, bv, n_kv, nullptr, false, [&](const float (&x)[VPL], int h, bool live) {
    const long long dr = cache_row(h, live);
    if constexpr (FMT == KVQ_F16) {
      put16(a.v_dst, x, dr);
    } else if constexpr (FMT == KVQ_K8V4) {
      float y[VPL];
#pragma unroll
      for (int e = 0; e < VPL; ++e) y[e] = x[e];
      wht_group<VPL, LPR>(y, lane);
      q4_lanes<HD, VPL>(y, dr, j, lane, static_cast<uint8_t*>(a.v_dst), a.vs_dst);
    } else {
      q8_lanes<HD, VPL, LPR>(x, dr, j, static_cast<int8_t*>(a.v_dst), a.vs_dst);
    }
  });
}

template <int FMT, int HD, int T>
cudaError_t launch(RotaryArgs a, int sms, cudaStream_t s) {
  constexpr int RPW = 32 / (HD / VPL);
  const int nb = (a.n_q + RPW - 1) / RPW + 2 * ((a.pool.n_kv + RPW - 1) / RPW);
  // one CTA a token, or for few tokens as many as fill the SMs, down to one head
  // block a warp
  const int most = (nb + kRotWarps - 1) / kRotWarps;
  const long long fill = (long long)sms * kRotCtas / a.n_tok, want = fill > 1 ? fill : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.n_tok, (unsigned)(want < most ? want : most));
  const int n_parts = (int)cfg.gridDim.y * kRotWarps, qb = (a.n_q + RPW - 1) / RPW, kb = (a.pool.n_kv + RPW - 1) / RPW;
  a.mod_k = qb % n_parts;
  a.mod_v = (qb + kb) % n_parts;
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
