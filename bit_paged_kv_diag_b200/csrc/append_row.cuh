// append_row.cuh -- one K or V row held by a pair of lanes: the block-diagonal Hadamard
// butterfly and the INT4 / NVFP4 quantisers, shared by the append kernels.  Lane l of a row
// (l = 0, 1) holds channels [64l, 64l + 64) as 8 chunks of 8, chunk t ^ rho in register
// slot t (rho = lane & 7, or any value with rho & 1 = l); the append kernel's header derives
// the layout and the rounding rules.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "kvq_ptx.cuh"

namespace kvq {

constexpr float kMagic = 12582912.0f;          // 1.5 * 2^23

// Two fp32 values in one 64-bit register (low half = the even channel).
typedef unsigned long long f2;

__device__ __forceinline__ f2 pk(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void upk(f2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 sub2(f2 a, f2 b) {
  f2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// a * b + c per half, one rounding each.
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// fp16 bits -> fp32, exact (h + -0.0 keeps signed zeros).
__device__ __forceinline__ float cvt_f16(uint32_t h) {
  float d;
  asm("add.rn.f32.f16 %0, %1, %2;" : "=f"(d) : "h"(static_cast<uint16_t>(h)), "f"(-0.0f));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Stages h = 2 .. b/2 of the butterfly on a lane's half row, in rotate_row's register layout.
template <int BLOCK>
__device__ __forceinline__ void rotate_stages(int rho, int l, unsigned pmask, f2 (&x)[32]) {
  if constexpr (BLOCK > 1) {
    // Stages h = 2 (pair index e <-> e + 1) and h = 4 (e <-> e + 2) inside each chunk.
#pragma unroll
    for (int t = 0; t < 8; t++)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const f2 a = x[4 * t + e], c = x[4 * t + e + 1];
        x[4 * t + e] = add2(a, c);
        x[4 * t + e + 1] = sub2(a, c);
      }
#pragma unroll
    for (int t = 0; t < 8; t++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const f2 a = x[4 * t + e], c = x[4 * t + e + 2];
        x[4 * t + e] = add2(a, c);
        x[4 * t + e + 2] = sub2(a, c);
      }
    // Stages h = 8, 16, 32: chunk bit k, slots t and t ^ (1 << k).  With bit k of rho
    // clear slot t holds the lower chunk: (t, u) <- (t + u, t - u); set: (u, t) <- (u + t,
    // u - t).  Both as fma(own, sg, other), sg = +-1.
#pragma unroll
    for (int k = 0; k < 3; k++) {
      if ((8 << k) < BLOCK) {
        const float sg = ((rho >> k) & 1) ? -1.0f : 1.0f;
        const f2 SG = pk(sg, sg), NSG = pk(-sg, -sg);
#pragma unroll
        for (int t = 0; t < 8; t++) {
          if (t & (1 << k)) continue;
          const int u = t | (1 << k);
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const f2 a = x[4 * t + e], c = x[4 * u + e];
            x[4 * t + e] = fma2(a, SG, c);
            x[4 * u + e] = fma2(c, NSG, a);
          }
        }
      }
    }
    if constexpr (BLOCK == 128) {
      // Stage h = 64 across the lane pair.  Lane 0's slot t and lane 1's slot t ^ 1 hold
      // the same chunk of their halves (rho differs in bit 0 between them), so every lane
      // receives its partner's slot t ^ 1 for its slot t.  Lane 0 (the lower channel)
      // keeps own + other, lane 1 (the upper) other - own: fma(own, +-1, other).
      const float sg = l ? -1.0f : 1.0f;
      const f2 SG = pk(sg, sg);
#pragma unroll
      for (int t = 0; t < 8; t += 2)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          float a0, a1, c0, c1;
          upk(x[4 * t + e], a0, a1);
          upk(x[4 * (t + 1) + e], c0, c1);
          const f2 ra = pk(__shfl_xor_sync(pmask, c0, 1), __shfl_xor_sync(pmask, c1, 1));
          const f2 rc = pk(__shfl_xor_sync(pmask, a0, 1), __shfl_xor_sync(pmask, a1, 1));
          x[4 * t + e] = fma2(x[4 * t + e], SG, ra);
          x[4 * (t + 1) + e] = fma2(x[4 * (t + 1) + e], SG, rc);
        }
    }
  }
}

// The butterfly without its final scale: x = z, the rotated row being y = fl(c_b * z),
// which quantise() applies where it needs y itself.  raw[t] = chunk t ^ rho of this lane's
// half row (4 words = 8 fp16 channels); x[4t + e] = channels 2e, 2e + 1 of that chunk.
template <int BLOCK>
__device__ __forceinline__ void rotate_row(const uint4 (&raw)[8], int rho, int l, unsigned pmask,
                                           f2 (&x)[32]) {
#pragma unroll
  for (int t = 0; t < 8; t++) {
    const uint32_t w[4] = {raw[t].x, raw[t].y, raw[t].z, raw[t].w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
      if constexpr (BLOCK == 1) {
        // b = 1 (plain INT4): the transform of size 1 is the identity and c_b = 1.
        x[4 * t + e] = pk(cvt_f16(w[e] & 0xffffu), cvt_f16(w[e] >> 16));
      } else {
        // Stage h = 1 fused with the conversion: (a, c) -> (a + c, a - c).
        const float c = cvt_f16(w[e] >> 16);
        const uint16_t lo = static_cast<uint16_t>(w[e] & 0xffffu);
        float s, d;
        asm("add.rn.f32.f16 %0, %1, %2;" : "=f"(s) : "h"(lo), "f"(c));
        asm("sub.rn.f32.f16 %0, %1, %2;" : "=f"(d) : "h"(lo), "f"(c));
        x[4 * t + e] = pk(s, d);
      }
    }
  }
  rotate_stages<BLOCK>(rho, l, pmask, x);
}

// The 8 codes of one chunk from their magic-rounded values (code = low nibble of the
// bits), packed low nibble = even channel.
__device__ __forceinline__ uint32_t pack_chunk(const f2 (&m)[4]) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; e++) upk(m[e], v[2 * e], v[2 * e + 1]);
  const uint32_t ev = prmt(prmt(__float_as_uint(v[0]), __float_as_uint(v[2]), 0x0040u),
                           prmt(__float_as_uint(v[4]), __float_as_uint(v[6]), 0x0040u), 0x5410u);
  const uint32_t od = prmt(prmt(__float_as_uint(v[1]), __float_as_uint(v[3]), 0x0040u),
                           prmt(__float_as_uint(v[5]), __float_as_uint(v[7]), 0x0040u), 0x5410u);
  uint32_t r;
  // (ev & 0x0F0F0F0F) | ((od << 4) & 0xF0F0F0F0)
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(ev), "r"(od << 4), "r"(0x0F0F0F0Fu));
  return r;
}

// Quantise this lane's 64 values of a row; q[t] = packed codes of slot t's chunk.
// Returns the fp16 scale bits (identical on both lanes of the row).
//
// Codes are round-half-even of y / s with s the stored fp16 scale.  Fast path (a normal,
// unsaturated s, so |y/s| <= 7.004): t = z * fl(c_b * fl(1/s)) (exact product) is within
// 4 roundings (< 2^-19) of y / s; fma(z, r_z, 1.5 * 2^23) rounds it to the nearest integer
// (ties to even) in one step, and fma(z, r_z, -rint) gives t - rint with one rounding, so
// the result is exact unless the fraction is within 2^-19 of one half.  A chunk with such
// a near-tie -- frequent for rows that are not rotated, whose fp16 values meet exact ties
// -- and every chunk when s is subnormal or saturated is recomputed exactly without
// dividing: k = floor(y*r) is within one of the true floor, and (k + 1/2)*s is exact in
// fp32 (an fp16 scale times a number of 5 bits), so comparing y with it chooses between k
// and k + 1, an exact tie going to the even one.  (If y*r fell on the wrong side of an
// integer n, y/s is within 2^-16 of n and both candidates' half points place it at n.)
// Codes are clamped to [-8, 7].
__device__ __forceinline__ uint16_t quantise(const f2 (&x)[32], float cb, unsigned pmask,
                                             uint32_t (&q)[8]) {
  // m = max |y| = fl(c_b * max |z|): rounding is monotonic, so scaling after the max gives
  // the max of the scaled values.
  float cm[8];  // per chunk, then a tree: short dependency chains
#pragma unroll
  for (int t = 0; t < 8; t++) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; e++) upk(x[4 * t + e], v[2 * e], v[2 * e + 1]);
    cm[t] = max3(max3(fabsf(v[0]), fabsf(v[1]), fabsf(v[2])),
                 max3(fabsf(v[3]), fabsf(v[4]), fabsf(v[5])), fmaxf(fabsf(v[6]), fabsf(v[7])));
  }
  float zmax = max3(max3(cm[0], cm[1], cm[2]), max3(cm[3], cm[4], cm[5]), fmaxf(cm[6], cm[7]));
  zmax = fmaxf(zmax, __shfl_xor_sync(pmask, zmax, 1));
  const float m = __fmul_rn(cb, zmax);
  const float s32 = __fdiv_rn(m, 7.0f);
  const bool sat = s32 > 65504.0f;
  const __half sh = sat ? __ushort_as_half(0x7BFF) : __float2half_rn(s32);
  const float s = __half2float(sh);
  if (s == 0.0f) {  // an all-zero row (or a scale that underflows): every code is 0
#pragma unroll
    for (int t = 0; t < 8; t++) q[t] = 0u;
    return __half_as_ushort(sh);
  }
  const bool normal = !sat && s >= 6.103515625e-05f;
  const float r = __frcp_rn(s);
  const float rz = __fmul_rn(cb, r);
  const float hs = 0.5f * s;
  const f2 MM = pk(kMagic, kMagic);
  const f2 RZ = pk(rz, rz);
  // Fast path for 4 chunks at a time, without branches; chunks with a near-tie are marked
  // and then recomputed exactly (rare for rotated rows).
#pragma unroll
  for (int g = 0; g < 8; g += 4) {
    uint32_t redo = normal ? 0u : 0xFFu;
#pragma unroll
    for (int t = g; t < g + 4; t++) {
      f2 mg[4];
      float d[8];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        mg[e] = fma2(x[4 * t + e], RZ, MM);   // 1.5*2^23 + rint(t)
        const f2 nr = sub2(MM, mg[e]);        // -rint(t), exactly
        upk(fma2(x[4 * t + e], RZ, nr), d[2 * e], d[2 * e + 1]);  // t - rint(t)
      }
      const float dmax = max3(max3(fabsf(d[0]), fabsf(d[1]), fabsf(d[2])),
                              max3(fabsf(d[3]), fabsf(d[4]), fabsf(d[5])), fmaxf(fabsf(d[6]), fabsf(d[7])));
      if (!(dmax < 0.5f - 0x1p-19f)) redo |= 1u << t;
      q[t] = pack_chunk(mg);
    }
    if (redo) {
#pragma unroll
      for (int t = g; t < g + 4; t++) {
        if (!((redo >> t) & 1u)) continue;
        f2 mg[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          float z[2], o[2];
          upk(x[4 * t + e], z[0], z[1]);
#pragma unroll
          for (int i = 0; i < 2; i++) {
            const float y = __fmul_rn(z[i], cb);  // the rotated value
            const float k = floorf(__fmul_rn(y, r));
            const float h = __fmaf_rn(k, s, hs);  // (k + 1/2) * s, exact
            const bool odd = (__float_as_uint(__fadd_rn(k, kMagic)) & 1u) != 0u;
            const bool up = y > h || (y == h && odd);
            const float c = fminf(fmaxf(up ? k + 1.0f : k, -8.0f), 7.0f);
            o[i] = __fadd_rn(c, kMagic);
          }
          mg[e] = pk(o[0], o[1]);
        }
        q[t] = pack_chunk(mg);
      }
    }
  }
  return __half_as_ushort(sh);
}

// Two fp32 values -> one byte of E2M1 codes (lo -> low nibble), nearest even, saturating.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 q;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %1, %2;\n\tcvt.u32.u8 %0, q;\n\t}"
      : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp32 values -> two E4M3 bytes (lo -> low byte), nearest even, saturating at 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two E4M3 bytes (low 16 bits) -> their values (exact).
__device__ __forceinline__ float2 e4m3x2_value(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// NVFP4 quantisation of this lane's 64 values: q[t] = the 4 code bytes of slot t's chunk;
// returns the lane's 4 scale bytes in block order (byte m = block 4l + m of the row).
__device__ __forceinline__ uint32_t quantise_fp4(const f2 (&x)[32], float cb, int rho,
                                                uint32_t (&q)[8]) {
  const f2 CB = pk(cb, cb);
  float sv[4];
  uint32_t sb[4];
#pragma unroll
  for (int u = 0; u < 4; u++) {  // slot pair (2u, 2u + 1) = one block of 16 channels
    float v[16];
#pragma unroll
    for (int e = 0; e < 8; e++) upk(x[8 * u + e], v[2 * e], v[2 * e + 1]);
    const float m8a = max3(max3(fabsf(v[0]), fabsf(v[1]), fabsf(v[2])),
                           max3(fabsf(v[3]), fabsf(v[4]), fabsf(v[5])), fmaxf(fabsf(v[6]), fabsf(v[7])));
    const float m8b = max3(max3(fabsf(v[8]), fabsf(v[9]), fabsf(v[10])),
                           max3(fabsf(v[11]), fabsf(v[12]), fabsf(v[13])), fmaxf(fabsf(v[14]), fabsf(v[15])));
    // max |y| = fl(c_b * max |z|) (rounding is monotonic)
    sv[u] = __fdiv_rn(__fmul_rn(cb, fmaxf(m8a, m8b)), 6.0f);
  }
  const uint32_t s01 = e4m3x2(sv[0], sv[1]), s23 = e4m3x2(sv[2], sv[3]);
  sb[0] = s01 & 0xFFu;
  sb[1] = s01 >> 8;
  sb[2] = s23 & 0xFFu;
  sb[3] = s23 >> 8;
  const float2 f01 = e4m3x2_value(s01), f23 = e4m3x2_value(s23);
  const float sf[4] = {f01.x, f01.y, f23.x, f23.y};
#pragma unroll
  for (int u = 0; u < 4; u++) {
    const float r = sf[u] != 0.0f ? __frcp_rn(sf[u]) : 0.0f;
    const f2 R = pk(r, r);
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int t = 2 * u + h;
      uint32_t w = 0;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        float a, b;
        upk(mul2(mul2(x[4 * t + e], CB), R), a, b);  // t = fl(fl(z * c_b) * r)
        w |= e2m1x2(a, b) << (8 * e);
      }
      q[t] = sf[u] != 0.0f ? w : 0u;  // a zero scale: every code 0
    }
  }
  // Byte u of the word belongs to block (2u ^ rho) >> 1 = u ^ (rho >> 1) of the lane's half.
  const uint32_t words = sb[0] | (sb[1] << 8) | (sb[2] << 16) | (sb[3] << 24);
  const uint32_t r2 = static_cast<uint32_t>(rho >> 1);
  const uint32_t sel = (0u ^ r2) | ((1u ^ r2) << 4) | ((2u ^ r2) << 8) | ((3u ^ r2) << 12);
  return prmt(words, 0u, sel);
}

}  // namespace kvq
