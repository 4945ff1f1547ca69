// kvq_quant.cuh -- the cache formats' quantisers: int8 group scales and codes,
// K8V4's 4-bit codes, and rows of them held by groups of lanes (shared by
// the appends).  Bit-exact with the definitions in kvq.h; kvq_append.cu says
// why the multiplies used here give the same bits as the divisions.
#pragma once

#include "kvq_internal.cuh"
#include "kvq_ptx.cuh"

namespace kvq {
namespace {

// The group scale fp16_rne(fl32(a / 127)) from a multiply: y = a * fl(1/127)
// is within 2 fp32 ulps of fl32(a / 127), so the two round to the same fp16
// value unless an fp16 rounding midpoint (13 discarded bits equal to 0x1000)
// lies within that distance, or the result leaves the fp16 normal range;
// only then is the quotient itself computed.
__device__ __forceinline__ __half group_scale(float a) {
  const float y = a * (1.0f / 127.0f);
  const uint32_t low = __float_as_uint(y) & 0x1fffu;
  const bool exact_needed = (low > 0x1000u - 4u && low < 0x1000u + 4u) || !(y >= 6.103515625e-05f) ||
                            !(y < 65504.0f);
  return __float2half_rn(exact_needed ? a / 127.0f : y);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Packed fp32 pairs (two lanes of work per instruction).
__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
  return ((unsigned long long)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ float lo2(unsigned long long v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(unsigned long long v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long sub2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// The int8 code clamp(rint(x / sf), -127, 127) from the IEEE fp32 quotient
// itself, as a byte (0 for a zero scale or a NaN quotient).
__device__ __forceinline__ uint32_t exact_code(float x, float sf) {
  if (sf == 0.0f) return 0u;
  const float qv = x / sf;
  if (!(qv == qv)) return 0u;
  return (uint32_t)(int)fminf(fmaxf(rintf(qv), -127.0f), 127.0f) & 0xffu;
}

// Codes of 4 values of one group (finite group maximum, so x is finite), as
// 4 bytes.  y = x * rs (rs = 1 / sf within one ulp) is within 2^-21 |x / sf|
// of the real quotient, and |x / sf| < 256, so wherever y lies more than
// 2.5e-4 from a half-integer the real quotient, its fp32 rounding and y
// round to the same integer; only inside that band are the quotients
// themselves used.  After clamping y to [-127, 127], y + 1.5 * 2^23 rounds y
// to an integer (to nearest, ties to even) in the low mantissa bits, whose
// low byte is the two's-complement code.
__device__ __forceinline__ uint32_t codes4(const float4& x, float sf, float rs) {
  if (sf == 0.0f) return 0u;
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  const unsigned long long r2 = pack2(rs, rs), m2 = pack2(kMagic, kMagic);
  const unsigned long long p01 = mul2(pack2(x.x, x.y), r2), p23 = mul2(pack2(x.z, x.w), r2);
  const unsigned long long y01 = pack2(fminf(fmaxf(lo2(p01), -127.0f), 127.0f),
                                       fminf(fmaxf(hi2(p01), -127.0f), 127.0f));
  const unsigned long long y23 = pack2(fminf(fmaxf(lo2(p23), -127.0f), 127.0f),
                                       fminf(fmaxf(hi2(p23), -127.0f), 127.0f));
  const unsigned long long t01 = add2(y01, m2), t23 = add2(y23, m2);
  const unsigned long long d01 = sub2(y01, sub2(t01, m2)), d23 = sub2(y23, sub2(t23, m2));
  constexpr float kBand = 0.5f - 2.5e-4f;
  const bool tie = fabsf(lo2(d01)) > kBand || fabsf(hi2(d01)) > kBand || fabsf(lo2(d23)) > kBand ||
                   fabsf(hi2(d23)) > kBand;
  if (tie)  // near a tie: the quotients decide (a few groups in a thousand)
    return exact_code(x.x, sf) | (exact_code(x.y, sf) << 8) | (exact_code(x.z, sf) << 16) |
           (exact_code(x.w, sf) << 24);
  return prmt(prmt((uint32_t)t01, (uint32_t)(t01 >> 32), 0x0040u),
              prmt((uint32_t)t23, (uint32_t)(t23 >> 32), 0x0040u), 0x5410u);
}

// K8V4 V codes of U values y of one block of scale d: the 4-bit offset
// codes clamp(rint(y / d), -8, 7) + 8, packed 4 bits each (value e in bits
// 4e..4e+3).  |y / d| <= 8 (up to d's fp16 rounding), so y * rs (rs ~ 1/d)
// is within 2e-6 of the quotient and decides the integer wherever it lies
// more than 2.5e-4 from a half-integer; adding and taking off 1.5 * 2^23
// rounds it (to nearest even) in packed pairs.  If any of the U values
// lies inside that band, or is not finite, the IEEE quotients decide all
// U (a NaN quotient gives 0).  Clamping to integer bounds commutes with
// rounding; the clamped integer k plus 1.5 * 2^23 + 8 has k + 8 in its
// low mantissa bits.  d == 0 gives code 8 throughout.
template <int U>
__device__ __forceinline__ uint32_t q4_codes(const float (&y)[U], float d) {
  if (d == 0.0f) return U == 4 ? 0x8888u : 0x88u;
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  constexpr float kBand = 0.5f - 2.5e-4f;
  const float rs = rcp_approx(d);
  const unsigned long long r2 = pack2(rs, rs), m2 = pack2(kMagic, kMagic);
  float k[U];
  bool near = false;
#pragma unroll
  for (int e = 0; e < U; e += 2) {
    const unsigned long long qa = mul2(pack2(y[e], y[e + 1]), r2);
    const unsigned long long r = sub2(add2(qa, m2), m2);
    const unsigned long long df = sub2(qa, r);
    near |= !(fabsf(lo2(df)) < kBand) || !(fabsf(hi2(df)) < kBand);
    k[e] = lo2(r);
    k[e + 1] = hi2(r);
  }
  if (near) {  // rare: the quotients themselves
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const float r = rintf(__fdiv_rn(y[e], d));
      k[e] = r == r ? r : 0.0f;
    }
  }
  uint32_t out = 0;
#pragma unroll
  for (int e = 0; e < U; ++e)
    out |= (__float_as_uint(fminf(fmaxf(k[e], -8.0f), 7.0f) + (kMagic + 8.0f)) & 15u) << (4 * e);
  return out;
}

// Lane-group row shape of the bulk int8 and K8V4 appends: a row (one token
// and KV head, K and V) is held by a group of LPR consecutive lanes, lane j
// of the group holding the VPL consecutive dims j VPL .. j VPL + VPL - 1
// (64 contiguous bytes of fp32 at VPL 16), so a warp carries 32 / LPR rows
// at once.  Bulk appends take VPL = 16 (8 at HD 64): few shuffles per row;
// a few K8V4 rows (decode steps) take VPL = 4 (8 at HD 256): short chains.
template <int HD, int VPL_>
struct LaneRows {
  static constexpr int VPL = VPL_;                // values a lane holds (4, 8 or 16)
  static constexpr int LPR = HD / VPL;            // lanes of a row
  static constexpr int RPW = 32 / LPR;            // rows a warp holds
  static_assert(VPL % 4 == 0 && LPR <= 32 && LPR * VPL == HD, "K8V4 row shape");
};

// int8 codes of one row held by a lane group (LaneRows layout): the group
// maximum over the 64 / VPL lanes of each 64-dim group (bit patterns of |x|,
// as the int8 kernel), group_scale, codes4 (or the quotients for a
// non-finite group); dr < 0 stores nothing.
template <int HD, int VPL, int LPR>
__device__ __forceinline__ void q8_lanes(const float (&x)[VPL], long long dr, int j, int8_t* codes,
                                         __half* scales) {
  constexpr int NG = HD / kGroup;
  constexpr int LG = kGroup / VPL;  // lanes of a 64-dim group
  uint32_t mb = 0;
#pragma unroll
  for (int e = 0; e < VPL; ++e) mb = max(mb, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
  for (int off = 1; off < LG; off <<= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, off));
  const float amax = __uint_as_float(mb);
  const __half sh = group_scale(amax);
  const float sf = __half2float(sh);
  uint32_t c[VPL / 4];
  if (amax <= 3.4028234663852886e38f) {
    const float rs = rcp_approx(sf);
#pragma unroll
    for (int q = 0; q < VPL / 4; ++q)
      c[q] = codes4(make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]), sf, rs);
  } else {
#pragma unroll
    for (int q = 0; q < VPL / 4; ++q)
      c[q] = exact_code(x[4 * q], sf) | (exact_code(x[4 * q + 1], sf) << 8) |
             (exact_code(x[4 * q + 2], sf) << 16) | (exact_code(x[4 * q + 3], sf) << 24);
  }
  if (dr >= 0) {
    int8_t* dst = codes + dr * HD + j * VPL;
    if constexpr (VPL == 16)
      *reinterpret_cast<uint4*>(dst) = make_uint4(c[0], c[1], c[VPL > 8 ? 2 : 0], c[VPL > 8 ? 3 : 0]);
    else if constexpr (VPL == 8)
      *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[VPL > 4 ? 1 : 0]);
    else
      *reinterpret_cast<uint32_t*>(dst) = c[0];
    if (j % LG == 0) scales[dr * NG + (j * VPL) / kGroup] = sh;
  }
}

// 4-bit codes of one rotated V row held by a lane group (LaneRows layout): per
// block of 32 dims the element of largest magnitude, the first one on ties
// (NaN counts as 0, a zero maximum gives m = +0), d = fp16(m / -8), two codes
// a byte; dr < 0 stores nothing.
template <int HD, int VPL>
__device__ __forceinline__ void q4_lanes(const float (&y)[VPL], long long dr, int j, int lane, uint8_t* codes,
                                         __half* scales) {
  constexpr int NB = HD / kQ4Block;
  constexpr int LB = kQ4Block / VPL;  // lanes of a 32-dim V block
  // the block's largest |y| (fmaxf drops NaN, so NaN counts as 0) ...
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < VPL; ++e) amax = fmaxf(amax, fabsf(y[e]));
#pragma unroll
  for (int off = 1; off < LB; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  // ... and the first dim holding it: the lowest lane of the block with a
  // match (lanes hold ascending dims), then its lowest element (the
  // backward scan keeps the lowest)
  float mine = 0.f;
  bool found = false;
#pragma unroll
  for (int e = VPL - 1; e >= 0; --e)
    if (fabsf(y[e]) == amax) {
      mine = y[e];
      found = true;
    }
  const unsigned blk_lanes = ((1u << LB) - 1u) << (lane & ~(LB - 1));
  const unsigned hit = __ballot_sync(0xffffffffu, found) & blk_lanes;
  const int src = hit ? __ffs(hit) - 1 : lane;  // no match only if amax is 0 (all NaN)
  float m = __shfl_sync(0xffffffffu, mine, src);
  if (amax == 0.f) m = 0.0f;  // no nonzero element: m stays +0
  const __half dh = __float2half_rn(m * -0.125f);  // = m / -8, both correctly rounded
  const float d = __half2float(dh);
  uint32_t c[VPL / 4];  // 4 codes (16 bits) each; dims 2i low nibble, 2i + 1 high
#pragma unroll
  for (int q = 0; q < VPL / 4; ++q) {
    const float y4[4] = {y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]};
    c[q] = q4_codes<4>(y4, d);
  }
  if (dr >= 0) {
    uint8_t* dst = codes + dr * (HD / 2) + j * (VPL / 2);
    if constexpr (VPL == 16)
      *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | (c[1] << 16), c[VPL > 8 ? 2 : 0] | (c[VPL > 8 ? 3 : 0] << 16));
    else if constexpr (VPL == 8)
      *reinterpret_cast<uint32_t*>(dst) = c[0] | (c[VPL > 4 ? 1 : 0] << 16);
    else
      *reinterpret_cast<uint16_t*>(dst) = (uint16_t)c[0];
    if (j % LB == 0) scales[dr * NB + (j * VPL) / kQ4Block] = dh;
  }
}

}  // namespace
}  // namespace kvq
