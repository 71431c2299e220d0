// The block-scaled 8-bit cache's number formats: one power-of-two scale for
// the 16 rows of a page, codes in E4M3 or int8, value = code * scale.
//
// A set of bf16 values whose largest finite magnitude is a gets the smallest
// power of two s = 2^e, e >= -126, with a <= max * s (max = 448 for E4M3, 127
// for int8), or 0 when a is 0. Why a power of two: x / s is exact, so a code is
// rounded once; and when a page's scale has to grow for a new row, the codes
// before it are multiplied by a power of two, which E4M3 takes exactly (but for
// values that become subnormal) and which costs int8 at most half a step of
// each new scale, one step in all however often the scale grows (the steps at
// least double each time). An arbitrary scale would use up to one bit more of
// int8's range and lose half a step at every growth.
#pragma once

#include <atomic>

#include <cuda_fp16.h>

#include "kvp_common.cuh"

namespace kvp {
namespace {

// Loads of data that the launch before may have written. The kernels of this cache start early behind that launch and
// wait for it on the device, so what they read must not be taken for constant while they run: a read-only load
// (__ldg, or a const __restrict__ parameter) may be served from a first-level line older than that launch, and the
// compiler may move it ahead of the wait. Hence no __restrict__ on what these kernels read, plain loads where nothing
// else is said, and these, which stay in order with the wait. For the same reason the last kernel of a call does not
// let its dependents start before it ends: they may be kernels that read what it writes with read-only loads.
KVP_DEV uint4 load16_stream(const void* p) {  // read once: first to leave the caches
  uint4 r;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
KVP_DEV float4 load16_l2(const void* p) {  // other CTAs' results, from L2
  float4 r;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "l"(p) : "memory");
  return r;
}
KVP_DEV float2 load8_l2(const void* p) {
  float2 r;
  asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(r.x), "=f"(r.y) : "l"(p) : "memory");
  return r;
}

// The scale (fp32 bits) for largest magnitude `a`, given as finite bf16 bits
// without the sign. With a = 2^(E - 127) (1 + f / 128): E4M3's largest number is
// 2^8 * 1.75 (f = 96), int8's 2^6 * (1 + 126 / 128).
template <int FMT>
KVP_DEV uint32_t scale_bits_for(uint32_t a) {
  if (a == 0) return 0u;
  const int E = static_cast<int>(a >> 7), f = static_cast<int>(a & 127u);
  const int e = FMT == KVP_BLOCK8_E4M3 ? E - 8 + (f > 96) : E - 6 + (f > 126);
  return static_cast<uint32_t>(max(e, 1)) << 23;
}

// 1 / s of a scale (1 for 0: the finite values are zeros); s is at most 2^122, so the inverse is normal.
KVP_DEV float inverse_of_scale(uint32_t bits) { return bits == 0 ? 1.f : __uint_as_float((254u << 23) - bits); }

// Magnitudes of two packed bf16 values, those that are not finite as 0.
KVP_DEV uint32_t finite_abs2(uint32_t w) {
  const uint32_t a = w & 0x7FFF7FFFu;
  return a & ~__vcmpgeu2(a, 0x7F807F80u);
}

// Two values, already divided by their scale, to codes in the low 16 bits (the
// first in the low byte): rounded to nearest even; infinities saturate, a NaN
// becomes E4M3's NaN, or 0 in int8.
template <int FMT>
KVP_DEV uint32_t encode2(float lo, float hi) {
  if constexpr (FMT == KVP_BLOCK8_E4M3) {
    return cvt_f32x2_to_e4m3x2(lo, hi);
  } else {
    const int a = min(max(__float2int_rn(lo), -127), 127), b = min(max(__float2int_rn(hi), -127), 127);
    return (static_cast<uint32_t>(a) & 0xFFu) | ((static_cast<uint32_t>(b) & 0xFFu) << 8);
  }
}
// Eight bf16 values (w, element 0 in the low half of w.x) times inv, to eight codes.
template <int FMT>
KVP_DEV uint2 encode8(const uint4& w, float inv) {
  uint2 r;
  r.x = encode2<FMT>(__fmul_rn(bf16_lo(w.x), inv), __fmul_rn(bf16_hi(w.x), inv)) |
        (encode2<FMT>(__fmul_rn(bf16_lo(w.y), inv), __fmul_rn(bf16_hi(w.y), inv)) << 16);
  r.y = encode2<FMT>(__fmul_rn(bf16_lo(w.z), inv), __fmul_rn(bf16_hi(w.z), inv)) |
        (encode2<FMT>(__fmul_rn(bf16_lo(w.w), inv), __fmul_rn(bf16_hi(w.w), inv)) << 16);
  return r;
}
// The same for values known to be finite (so that |x| * inv is at most the format's largest number). int8: adding
// 1.5 * 2^23 in the multiplication's own rounding leaves the rounded integer in the sum's low byte.
template <int FMT>
KVP_DEV uint2 encode8_finite(const uint4& w, float inv) {
  if constexpr (FMT == KVP_BLOCK8_E4M3) {
    return encode8<FMT>(w, inv);
  } else {
    auto four = [&](uint32_t a, uint32_t b) {
      const uint32_t x = __float_as_uint(fmaf(bf16_lo(a), inv, 12582912.f)), y = __float_as_uint(fmaf(bf16_hi(a), inv, 12582912.f));
      const uint32_t z = __float_as_uint(fmaf(bf16_lo(b), inv, 12582912.f)), u = __float_as_uint(fmaf(bf16_hi(b), inv, 12582912.f));
      return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, u, 0x0040), 0x5410);
    };
    return make_uint2(four(w.x, w.y), four(w.z, w.w));
  }
}

// The two codes in the low 16 bits of `two` as numbers, exactly.
template <int FMT>
KVP_DEV float2 decode2(uint32_t two) {
  if constexpr (FMT == KVP_BLOCK8_E4M3) {
    const uint32_t h2 = cvt_e4m3x2_to_f16x2(two);
    return __half22float2(*reinterpret_cast<const __half2*>(&h2));
  } else {
    return make_float2(static_cast<float>(static_cast<int8_t>(two & 0xFFu)),
                       static_cast<float>(static_cast<int8_t>((two >> 8) & 0xFFu)));
  }
}
// Four codes times `ratio` (a power of two, at most 1), rounded to codes again.
template <int FMT>
KVP_DEV uint32_t rescale4(uint32_t w, float ratio) {
  const float2 a = decode2<FMT>(w), b = decode2<FMT>(w >> 16);
  return encode2<FMT>(__fmul_rn(a.x, ratio), __fmul_rn(a.y, ratio)) |
         (encode2<FMT>(__fmul_rn(b.x, ratio), __fmul_rn(b.y, ratio)) << 16);
}

}  // namespace
}  // namespace kvp
