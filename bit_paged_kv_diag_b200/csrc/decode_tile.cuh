// decode_tile.cuh -- one 32-token tile of the 4-bit cache against one KV head's query group:
// the rotated q in fragment form, QK^T, softmax and PV steps of a warp, the warp's partial
// records and their merge.  Shared by the decode kernels; the decode kernel's header
// derives the layouts.
#pragma once

#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

namespace {

constexpr int kD = 128;
// Token row of a (page, head) block: codes, then scales (INT4: one fp16 per K/V row;
// NVFP4: one E4M3 per 16 channels), and the ring slot of one tile.
constexpr int row_bytes(bool fp4) { return fp4 ? kD + kD / 8 : kD + 4; }
constexpr int slot_bytes(bool fp4) { return kTileTokens * row_bytes(fp4); }
constexpr int kWarps = kDecodeWarps;                // warps per CTA
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;                          // ring slots per warp
constexpr uint64_t kWaitLimitNs = 2000000000ull;    // bounded waits: 2 s
constexpr unsigned kFull = 0xffffffffu;
constexpr float kMagic = 12582912.0f;               // 1.5 * 2^23

// ------------------------------------------------------------------------ q --
// int8 B fragments of the rotated, scaled q, per k32 chunk jj: [jj][0] = k 4c..4c+3,
// [jj][1] = k 16+4c..16+4c+3, where k = 4c + e <-> channel 32c + 8jj + 2e and
// k = 16 + 4c + e <-> channel 32c + 8jj + 2e + 1.
// G <= 4: A = column g holds slice 1 (g even) or 2 (g odd) of query g/2, B = slice 3
// (g even) or zero.  G == 8: A, B, C = slices 1, 2, 3 of query g.
template <int G>
struct QFrag {
  static constexpr int NQ = (G == 8) ? 2 : 1;  // queries owned by one thread
  uint32_t A[4][2], B[4][2], C[4][2];
  float sf[NQ];  // M / 1024 of the owned queries
};

// Rotate (the fixed-order butterfly: stages h = 1, 2 in registers, h = 4..64 across
// lanes), scale by c_b * softmax_scale * log2(e), and cut every query of the unit into
// three int8 slices q' = M/64 * (q1 + q2/128 + q3/16384), M the power of two >= max|q'|
// (1 for a zero row).  qraw: the unit's G fp16 rows in shared memory; the slices go to the
// warp's fragment table in fragment order:
//   frag word ((qi*3 + s)*4 + c)*8 + 2*jj + half, byte e  <->  channel 32c + 8jj + 2e + half.
// The warp prepares queries q0, q0 + QSTEP, ... < G (all of them for QSTEP = 1; a
// quarter each when the CTA's warps share one unit's rows).
// Rotated, scaled queries qb, qb + QSTEP, ... (QB of them; indices past G repeat the last
// one and are not stored by the callers): x[b][e] = channel 4*lane + e, and the power of
// two M[b] >= max |q'| (1 for a zero row).
template <int G, int QSTEP, int QB>
__device__ __forceinline__ void rotate_q(const uint8_t* qraw, int qb, int lane, const DecodeParams& p,
                                       float (&x)[QB][4], float (&M)[QB]) {
#pragma unroll
  for (int b = 0; b < QB; b++) {
    const int qi = min(qb + b * QSTEP, G - 1);  // a clamped duplicate is computed, not stored
    const uint2 raw = *reinterpret_cast<const uint2*>(qraw + qi * kD * 2 + 8 * lane);
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
    const float t0 = lo.x, t1 = lo.y, t2 = hi.x, t3 = hi.y;
    const float a0 = __fadd_rn(t0, t1), a1 = __fsub_rn(t0, t1);
    const float a2 = __fadd_rn(t2, t3), a3 = __fsub_rn(t2, t3);
    const bool rot = p.hadamard_block > 1;  // b = 1 (plain INT4): no rotation
    x[b][0] = rot ? __fadd_rn(a0, a2) : t0;
    x[b][2] = rot ? __fsub_rn(a0, a2) : t2;
    x[b][1] = rot ? __fadd_rn(a1, a3) : t1;
    x[b][3] = rot ? __fsub_rn(a1, a3) : t3;
  }
#pragma unroll
  for (int s = 0; s < 5; s++) {
    if ((4 << s) < p.hadamard_block) {
      const float sgn = ((lane >> s) & 1) ? -1.0f : 1.0f;
#pragma unroll
      for (int b = 0; b < QB; b++)
#pragma unroll
        for (int e = 0; e < 4; e++)
          x[b][e] = __fmaf_rn(x[b][e], sgn, __shfl_xor_sync(kFull, x[b][e], 1 << s));
    }
  }
  float amax[QB];
#pragma unroll
  for (int b = 0; b < QB; b++) {
    amax[b] = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      x[b][e] = __fmul_rn(__fmul_rn(x[b][e], p.cb), p.q_scale);
      amax[b] = fmaxf(amax[b], fabsf(x[b][e]));
    }
  }
#pragma unroll
  for (int d = 1; d < 32; d *= 2)
#pragma unroll
    for (int b = 0; b < QB; b++) amax[b] = fmaxf(amax[b], __shfl_xor_sync(kFull, amax[b], d));
#pragma unroll
  for (int b = 0; b < QB; b++) {
    M[b] = 1.0f;
    if (amax[b] > 1e-30f) {
      const uint32_t bits = __float_as_uint(amax[b]);
      M[b] = (bits & 0x7FFFFFu) ? __uint_as_float((bits & 0x7F800000u) + 0x00800000u) : amax[b];
    }
  }
}

template <int G, int QSTEP>
__device__ __forceinline__ void prep_q_warp(const uint8_t* qraw, uint32_t* frag, float* sf, int lane,
                                            const DecodeParams& p, int q0 = 0) {
  // Up to four queries at a time: their shuffle chains are independent and interleave.
  constexpr int NQW = (G + QSTEP - 1) / QSTEP;
  constexpr int QB = NQW < 4 ? NQW : 4;
  const int c = lane >> 3, jj = (lane >> 1) & 3, e0 = (2 * lane) & 3;
  uint8_t* base = reinterpret_cast<uint8_t*>(frag);
#pragma unroll 1
  for (int qb = q0; qb < G; qb += QB * QSTEP) {
    float x[QB][4];
#pragma unroll
    for (int b = 0; b < QB; b++) {
      const int qi = min(qb + b * QSTEP, G - 1);  // a clamped duplicate is computed, not stored
      const uint2 raw = *reinterpret_cast<const uint2*>(qraw + qi * kD * 2 + 8 * lane);
      const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
      const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
      const float t0 = lo.x, t1 = lo.y, t2 = hi.x, t3 = hi.y;
      const float a0 = __fadd_rn(t0, t1), a1 = __fsub_rn(t0, t1);
      const float a2 = __fadd_rn(t2, t3), a3 = __fsub_rn(t2, t3);
      const bool rot = p.hadamard_block > 1;  // b = 1 (plain INT4): no rotation
      x[b][0] = rot ? __fadd_rn(a0, a2) : t0;
      x[b][2] = rot ? __fsub_rn(a0, a2) : t2;
      x[b][1] = rot ? __fadd_rn(a1, a3) : t1;
      x[b][3] = rot ? __fsub_rn(a1, a3) : t3;
    }
#pragma unroll
    for (int s = 0; s < 5; s++) {
      if ((4 << s) < p.hadamard_block) {
        const float sgn = ((lane >> s) & 1) ? -1.0f : 1.0f;
#pragma unroll
        for (int b = 0; b < QB; b++)
#pragma unroll
          for (int e = 0; e < 4; e++)
            x[b][e] = __fmaf_rn(x[b][e], sgn, __shfl_xor_sync(kFull, x[b][e], 1 << s));
      }
    }
    float amax[QB];
#pragma unroll
    for (int b = 0; b < QB; b++) {
      amax[b] = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        x[b][e] = __fmul_rn(__fmul_rn(x[b][e], p.cb), p.q_scale);
        amax[b] = fmaxf(amax[b], fabsf(x[b][e]));
      }
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2)
#pragma unroll
      for (int b = 0; b < QB; b++) amax[b] = fmaxf(amax[b], __shfl_xor_sync(kFull, amax[b], d));
#pragma unroll
    for (int b = 0; b < QB; b++) {
      float M = 1.0f;
      if (amax[b] > 1e-30f) {
        const uint32_t bits = __float_as_uint(amax[b]);
        M = (bits & 0x7FFFFFu) ? __uint_as_float((bits & 0x7F800000u) + 0x00800000u) : amax[b];
      }
      const float inv = __fdiv_rn(64.0f, M);  // exact: powers of two
      uint32_t ms[3][4];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const float t = x[b][e] * inv;                      // |t| <= 64, exact scaling
        const float m1 = t + kMagic;                        // rint(t) in the low mantissa bits
        const float r1 = (t - (m1 - kMagic)) * 128.0f;      // exact
        const float m2 = r1 + kMagic;
        const float r2 = (r1 - (m2 - kMagic)) * 128.0f;
        const float m3 = r2 + kMagic;
        ms[0][e] = __float_as_uint(m1);
        ms[1][e] = __float_as_uint(m2);
        ms[2][e] = __float_as_uint(m3);
      }
      // Channels 4*lane + i: c = lane/8, jj = (lane/2)%4, half = i%2, byte e0 + i/2 with
      // e0 = (2*lane)%4: a 2-byte store per (slice, half).
      const int qi = qb + b * QSTEP;
      if (qi >= G) continue;
#pragma unroll
      for (int sl = 0; sl < 3; sl++) {
        const int word = ((qi * 3 + sl) * 4 + c) * 8 + 2 * jj;
        const uint16_t h0 = static_cast<uint16_t>((ms[sl][0] & 0xFFu) | ((ms[sl][2] & 0xFFu) << 8));
        const uint16_t h1 = static_cast<uint16_t>((ms[sl][1] & 0xFFu) | ((ms[sl][3] & 0xFFu) << 8));
        *reinterpret_cast<uint16_t*>(base + word * 4 + e0) = h0;
        *reinterpret_cast<uint16_t*>(base + (word + 1) * 4 + e0) = h1;
      }
      if (lane == 0) sf[qi] = M * (1.0f / 1024.0f);
    }
  }
  __syncwarp();
}

template <int G>
__device__ __forceinline__ void qfrag_load(QFrag<G>& f, const uint32_t* qfb, const float* sfb,
                                           int lane) {
  const int g = lane >> 2, c = lane & 3;
  const int qi = (G == 8) ? g : (g >> 1);
  const bool ok = qi < G;
  uint4 s[3][2];
#pragma unroll
  for (int sl = 0; sl < 3; sl++) {
    s[sl][0] = s[sl][1] = make_uint4(0u, 0u, 0u, 0u);
    if (ok) {
      const uint4* src = reinterpret_cast<const uint4*>(qfb + ((qi * 3 + sl) * 4 + c) * 8);
      s[sl][0] = src[0];
      s[sl][1] = src[1];
    }
  }
#pragma unroll
  for (int jj = 0; jj < 4; jj++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      uint32_t v[3];
#pragma unroll
      for (int sl = 0; sl < 3; sl++) {
        const uint4 q4 = s[sl][jj >> 1];
        const uint32_t wds[4] = {q4.x, q4.y, q4.z, q4.w};
        v[sl] = wds[2 * (jj & 1) + e];
      }
      if (G == 8) {
        f.A[jj][e] = v[0];
        f.B[jj][e] = v[1];
        f.C[jj][e] = v[2];
      } else {
        f.A[jj][e] = (g & 1) ? v[1] : v[0];
        f.B[jj][e] = (g & 1) ? 0u : v[2];
        f.C[jj][e] = 0u;
      }
    }
  if (G == 8) {
    f.sf[0] = sfb[2 * c];
    f.sf[QFrag<G>::NQ - 1] = sfb[2 * c + 1];
  } else {
    f.sf[0] = c < G ? sfb[c] : 1.0f;
  }
}

// ---------------------------------------------------------------- NVFP4 q --
// NVFP4 cache ("BitDecoding-FP4:FP4 KVキャッシュのネイティブ復号" (sns.style): E2M1 codes
// with an E4M3 scale per 16 channels).  K and V are dequantised to fp16 exactly (an E2M1
// value times an E4M3 scale has at most 6 significant bits and lies in [2^-10, 2688]);
// QK^T and PV run as mma.sync m16n8k16 f16 x f16 -> f32.  q' is normalised by M (the
// power of two >= max |q'|) to |q~| <= 2^14 and carried as fp16 hi + lo parts (about
// 2^-22 relative).  Fragment table row (qi, part) = 128 fp16 in channel order.
template <int G, int QSTEP>
__device__ __forceinline__ void prep_q4_warp(const uint8_t* qraw, uint32_t* frag, float* sf, int lane,
                                             const DecodeParams& p, int q0 = 0) {
  constexpr int NQW = (G + QSTEP - 1) / QSTEP;
  constexpr int QB = NQW < 4 ? NQW : 4;
  __half* base = reinterpret_cast<__half*>(frag);
#pragma unroll 1
  for (int qb = q0; qb < G; qb += QB * QSTEP) {
    float x[QB][4], Mq[QB];
    rotate_q<G, QSTEP, QB>(qraw, qb, lane, p, x, Mq);
#pragma unroll
    for (int b = 0; b < QB; b++) {
      const int qi = qb + b * QSTEP;
      if (qi >= G) continue;
      const float inv = __fdiv_rn(16384.0f, Mq[b]);  // exact: powers of two
      __half hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const float t = x[b][e] * inv;
        hi[e] = __float2half_rn(t);
        lo[e] = __float2half_rn(t - __half2float(hi[e]));
      }
      *reinterpret_cast<uint2*>(base + (qi * 2) * kD + 4 * lane) =
          make_uint2(pack_half2(hi[0], hi[1]), pack_half2(hi[2], hi[3]));
      *reinterpret_cast<uint2*>(base + (qi * 2 + 1) * kD + 4 * lane) =
          make_uint2(pack_half2(lo[0], lo[1]), pack_half2(lo[2], lo[3]));
      if (lane == 0) sf[qi] = Mq[b] * (1.0f / 16384.0f);
    }
  }
  __syncwarp();
}

// f16 B fragments of q~ per k-step kk (16 channels: k rows 2c + e <-> channel
// 32c + 4kk + e, k rows 2c + 8 + e <-> channel 32c + 4kk + 2 + e), column g.
// G <= 4: column g holds part g & 1 (hi, lo) of query g / 2 in H; G == 8: H and L are the
// hi and lo parts of query g.
template <int G>
struct QFrag4 {
  static constexpr int NQ = (G == 8) ? 2 : 1;
  uint32_t H[8][2];
  uint32_t L[G == 8 ? 8 : 1][2];
  float sf[NQ];
};

template <int G>
__device__ __forceinline__ void qfrag4_load(QFrag4<G>& f, const uint32_t* qfb, const float* sfb,
                                            int lane) {
  const int g = lane >> 2, c = lane & 3;
  const int qi = (G == 8) ? g : (g >> 1);
  const bool ok = qi < G;
  const int row_h = (G == 8) ? 2 * g : 2 * qi + (g & 1);
#pragma unroll
  for (int part = 0; part < (G == 8 ? 2 : 1); part++) {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (ok) w[i] = reinterpret_cast<const uint4*>(qfb + (row_h + part) * (kD / 2) + 16 * c)[i];
    }
#pragma unroll
    for (int kk = 0; kk < 8; kk++) {
      const uint4 q4 = w[kk >> 1];
      const uint32_t a = (kk & 1) ? q4.z : q4.x, b = (kk & 1) ? q4.w : q4.y;
      if (part == 0) {
        f.H[kk][0] = a;
        f.H[kk][1] = b;
      } else {
        f.L[G == 8 ? kk : 0][0] = a;
        f.L[G == 8 ? kk : 0][1] = b;
      }
    }
  }
  if (G == 8) {
    f.sf[0] = sfb[2 * c];
    f.sf[QFrag4<G>::NQ - 1] = sfb[2 * c + 1];
  } else {
    f.sf[0] = c < G ? sfb[c] : 1.0f;
  }
}

// The 4 bytes of w, each two E2M1 codes (low nibble first) -> 4 x fp16x2, exact.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&d)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(w));
}

// Two E4M3 scale bytes (low 16 bits, low byte first) -> fp16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Tokens to attend of each 16-token half of a tile (a prefix of the half; may be <= 0 or > 16).
struct Valid {
  int n[2];
};
// Whether token 16 j + tau of a tile is attended: of a tile with a valid prefix of ntok tokens, or
// with a prefix in each half.
__device__ __forceinline__ bool tok_valid(int ntok, int j, int tau) { return 16 * j + tau < ntok; }
__device__ __forceinline__ bool tok_valid(Valid v, int j, int tau) { return tau < v.n[j]; }

// Scores (log2 domain) of an NVFP4 tile, in tile_qk's layout: A row g <-> token tau0,
// row g + 8 <-> tau1; the lane's 16 code bytes of a token row are channels 32c..32c+31
// (blocks 2c, 2c + 1), byte 2kk <-> channels 32c + 4kk, +1 (k columns 2c, 2c + 1).
template <int G, int SEFF, typename N>
__device__ __forceinline__ void tile_qk4(const QFrag4<G>& qf, const uint8_t* slot, N ntok, int lane,
                                         float (&sc)[2][QFrag4<G>::NQ][2]) {
  constexpr int RB = row_bytes(true);
  const int g = lane >> 2, c = lane & 3;
  const int tau0 = (g < 4) ? g : g + 4;
  const int tau1 = tau0 + 4;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const uint8_t* pbase = slot + (16 * j / SEFF) * (SEFF * RB);
    const int sl = (16 * j) % SEFF;
    const uint4 ka = *reinterpret_cast<const uint4*>(pbase + (sl + tau0) * 64 + 16 * c);
    const uint4 kc = *reinterpret_cast<const uint4*>(pbase + (sl + tau1) * 64 + 16 * c);
    const uint32_t sa = *reinterpret_cast<const uint16_t*>(pbase + SEFF * 128 + (sl + tau0) * 8 + 2 * c);
    const uint32_t sc2 = *reinterpret_cast<const uint16_t*>(pbase + SEFF * 128 + (sl + tau1) * 8 + 2 * c);
    const uint32_t fa = e4m3x2_to_f16x2(sa), fc = e4m3x2_to_f16x2(sc2);
    const uint32_t sA[2] = {prmt(fa, fa, 0x1010u), prmt(fa, fa, 0x3232u)};
    const uint32_t sC[2] = {prmt(fc, fc, 0x1010u), prmt(fc, fc, 0x3232u)};
    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w};
    const uint32_t wc[4] = {kc.x, kc.y, kc.z, kc.w};
    float accH[4] = {0.0f, 0.0f, 0.0f, 0.0f}, accL[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int wi = 0; wi < 4; wi++) {  // word wi = k-steps 2wi, 2wi + 1
      uint32_t da[4], dc[4];
      e2m1x8_to_f16x2(wa[wi], da);
      e2m1x8_to_f16x2(wc[wi], dc);
      const int blk = wi >> 1;  // k-steps 0-3: block 2c; 4-7: block 2c + 1
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int kk = 2 * wi + h;
        const uint32_t a0 = hmul2(da[2 * h], sA[blk]), a2 = hmul2(da[2 * h + 1], sA[blk]);
        const uint32_t a1 = hmul2(dc[2 * h], sC[blk]), a3 = hmul2(dc[2 * h + 1], sC[blk]);
        mma_16816(accH, a0, a1, a2, a3, qf.H[kk][0], qf.H[kk][1]);
        if (G == 8) mma_16816(accL, a0, a1, a2, a3, qf.L[G == 8 ? kk : 0][0], qf.L[G == 8 ? kk : 0][1]);
      }
    }
    const bool v0 = tok_valid(ntok, j, tau0), v1 = tok_valid(ntok, j, tau1);
    if (G == 8) {
#pragma unroll
      for (int qq = 0; qq < 2; qq++)
#pragma unroll
        for (int r = 0; r < 2; r++) {
          const int e = 2 * r + qq;
          sc[j][qq][r] = (r ? v1 : v0) ? (accH[e] + accL[e]) * qf.sf[qq] : -CUDART_INF_F;
        }
    } else {
      // Column 2c = hi part, 2c + 1 = lo part of query c.
      sc[j][0][0] = v0 ? (accH[0] + accH[1]) * qf.sf[0] : -CUDART_INF_F;
      sc[j][0][1] = v1 ? (accH[2] + accH[3]) * qf.sf[0] : -CUDART_INF_F;
    }
  }
}

// ------------------------------------------------------------------- state --
template <int G>
struct State {
  static constexpr int NQ = QFrag<G>::NQ;
  float o[8][4];  // PV accumulators: m-tile i = channels 16g+2i (rows g) and 16g+2i+1
  float m[NQ];
  float l[NQ];
};

template <int G>
__device__ __forceinline__ void state_reset(State<G>& st) {
#pragma unroll
  for (int i = 0; i < 8; i++)
#pragma unroll
    for (int e = 0; e < 4; e++) st.o[i][e] = 0.0f;
#pragma unroll
  for (int qq = 0; qq < State<G>::NQ; qq++) {
    st.m[qq] = -CUDART_INF_F;
    st.l[qq] = 0.0f;
  }
}


// One tile = 2 k-steps of 16 tokens in a ring slot (a shared-memory pointer); ntok: the
// valid tokens of each.  The work is split in three so that the QK^T of the next tile and the
// PV of the current one sit in one straight-line block the compiler can interleave.

// Scores (log2 domain) of the tile: sc[k-step][owned query][row], -inf past them.
template <int G, int SEFF, typename N>
__device__ __forceinline__ void tile_qk(const QFrag<G>& qf, const uint8_t* slot, N ntok, int lane,
                                        float (&sc)[2][QFrag<G>::NQ][2]) {
  const int g = lane >> 2, c = lane & 3;
  const int tau0 = (g < 4) ? g : g + 4;  // token of A row g
  const int tau1 = tau0 + 4;             // token of A row g + 8
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const uint8_t* pbase = slot + (16 * j / SEFF) * (SEFF * 132);
    const int sl = (16 * j) % SEFF;
    const uint4 ka = *reinterpret_cast<const uint4*>(pbase + (sl + tau0) * 64 + 16 * c);
    const uint4 kc = *reinterpret_cast<const uint4*>(pbase + (sl + tau1) * 64 + 16 * c);
    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w};
    const uint32_t wc[4] = {kc.x, kc.y, kc.z, kc.w};
    int accA[4] = {0, 0, 0, 0}, accB[4] = {0, 0, 0, 0}, accC[4] = {0, 0, 0, 0};
#pragma unroll
    for (int jj = 0; jj < 4; jj++) {
      const uint32_t a0 = (wa[jj] << 4) & 0xF0F0F0F0u, a1 = (wc[jj] << 4) & 0xF0F0F0F0u;
      const uint32_t a2 = wa[jj] & 0xF0F0F0F0u, a3 = wc[jj] & 0xF0F0F0F0u;
      mma_16832_s8(accA, a0, a1, a2, a3, qf.A[jj][0], qf.A[jj][1]);
      mma_16832_s8(accB, a0, a1, a2, a3, qf.B[jj][0], qf.B[jj][1]);
      if (G == 8) mma_16832_s8(accC, a0, a1, a2, a3, qf.C[jj][0], qf.C[jj][1]);
    }
    const __half* skp = reinterpret_cast<const __half*>(pbase + SEFF * 128) + sl;
    const float sk0 = __half2float(skp[tau0]), sk1 = __half2float(skp[tau1]);
    const bool v0 = tok_valid(ntok, j, tau0), v1 = tok_valid(ntok, j, tau1);
    const float k14 = 1.0f / 16384.0f;
    if (G == 8) {
      // Column 2c = query 2c (qq 0), 2c+1 = query 2c+1 (qq 1); rows g (d0, d1), g+8 (d2, d3).
#pragma unroll
      for (int qq = 0; qq < 2; qq++)
#pragma unroll
        for (int r = 0; r < 2; r++) {
          const int e = 2 * r + qq;
          const float v = static_cast<float>(accA[e]) + static_cast<float>(accB[e] * 128 + accC[e]) * k14;
          sc[j][qq][r] = (r ? v1 : v0) ? v * ((r ? sk1 : sk0) * qf.sf[qq]) : -CUDART_INF_F;
        }
    } else {
      // Column 2c = slices 1 (A) and 3 (B) of query c, 2c+1 = slice 2 (A) of query c.
      const float va = static_cast<float>(accA[0]) + static_cast<float>(accA[1] * 128 + accB[0]) * k14;
      const float vc = static_cast<float>(accA[2]) + static_cast<float>(accA[3] * 128 + accB[2]) * k14;
      sc[j][0][0] = v0 ? va * (sk0 * qf.sf[0]) : -CUDART_INF_F;
      sc[j][0][1] = v1 ? vc * (sk1 * qf.sf[0]) : -CUDART_INF_F;
    }
  }
}

// Online softmax update with the tile's scores, in two parts.  The statistics part moves
// m and l to the tile's frame and turns sc into p = exp2(score - m); it leaves the o'
// accumulators alone, so it can run next to the previous tile's PV.  The rescale part
// then brings o' to the new frame (alpha = exp2(m_old - m_new)).
template <int G>
__device__ __forceinline__ bool tile_softmax_stats(State<G>& st, float (&sc)[2][QFrag<G>::NQ][2],
                                                   float (&alpha)[QFrag<G>::NQ]) {
  constexpr int NQ = State<G>::NQ;
  bool rescale = false;
#pragma unroll
  for (int qq = 0; qq < NQ; qq++) {
    float mx = fmaxf(fmaxf(sc[0][qq][0], sc[0][qq][1]), fmaxf(sc[1][qq][0], sc[1][qq][1]));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
    const float mnew = fmaxf(st.m[qq], mx);
    alpha[qq] = ex2_approx(st.m[qq] - mnew);
    rescale |= alpha[qq] != 1.0f;
    st.m[qq] = mnew;
    float ps = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int r = 0; r < 2; r++) {
        sc[j][qq][r] = ex2_approx(sc[j][qq][r] - mnew);
        ps += sc[j][qq][r];
      }
    st.l[qq] = st.l[qq] * alpha[qq] + ps;
  }
  return __any_sync(kFull, rescale);
}

template <int G>
__device__ __forceinline__ void tile_rescale(State<G>& st, const float (&alpha)[QFrag<G>::NQ]) {
  constexpr int NQ = State<G>::NQ;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    // G <= 4: columns 2c, 2c+1 are query c's hi and lo parts; G == 8: queries 2c, 2c+1.
    st.o[i][0] *= alpha[0];
    st.o[i][2] *= alpha[0];
    st.o[i][1] *= alpha[NQ - 1];
    st.o[i][3] *= alpha[NQ - 1];
  }
}

// (p0, p1) -> fp16 pairs hi = rn(p), lo = rn(p - hi): p carried to about 2^-22.
__device__ __forceinline__ void split_hi_lo(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(p0, p1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(p0 - f.x, p1 - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// PV of the tile with probabilities pr.  B fragment of thread (g, c): tokens c, c+4 (b0)
// and c+8, c+12 (b1) of the k-step for column g, taken from the lanes that scored them
// (rows c and c + 4 of the QK^T fragment).
template <int G, int SEFF, typename N>
__device__ __forceinline__ void tile_pv(State<G>& st, const uint8_t* slot, N ntok, int lane,
                                        const float (&pr)[2][QFrag<G>::NQ][2]) {
  const int g = lane >> 2, c = lane & 3;
  const int tau0 = (g < 4) ? g : g + 4;
  const int tau1 = tau0 + 4;
  const int srcA = 4 * c + (g >> 1);
  const int srcB = srcA + 16;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const uint8_t* pbase = slot + (16 * j / SEFF) * (SEFF * 132);
    const int sl = (16 * j) % SEFF;
    const uint8_t* vb = pbase + SEFF * 64 + sl * 64;
    const __half* svp = reinterpret_cast<const __half*>(pbase + SEFF * 130) + sl;
    const float sv0 = __half2float(svp[tau0]), sv1 = __half2float(svp[tau1]);
    const bool v0 = tok_valid(ntok, j, tau0), v1 = tok_valid(ntok, j, tau1);
    // P' = p * s_v carried as fp16 hi + lo (relative precision ~2^-22).
    uint32_t bh0, bh1, bl0 = 0u, bl1 = 0u;
    if (G == 8) {
      uint32_t xh[2], xl[2];
#pragma unroll
      for (int qq = 0; qq < 2; qq++) {
        const float p0 = v0 ? pr[j][qq][0] * sv0 : 0.0f, p1 = v1 ? pr[j][qq][1] * sv1 : 0.0f;
        split_hi_lo(p0, p1, xh[qq], xl[qq]);
      }
      // Column g = query g, owned by lane group c' = g/2 as its query (g & 1).
      const uint32_t aE = __shfl_sync(kFull, xh[0], srcA), aO = __shfl_sync(kFull, xh[1], srcA);
      const uint32_t cE = __shfl_sync(kFull, xh[0], srcB), cO = __shfl_sync(kFull, xh[1], srcB);
      const uint32_t dE = __shfl_sync(kFull, xl[0], srcA), dO = __shfl_sync(kFull, xl[1], srcA);
      const uint32_t eE = __shfl_sync(kFull, xl[0], srcB), eO = __shfl_sync(kFull, xl[1], srcB);
      bh0 = (g & 1) ? aO : aE;
      bh1 = (g & 1) ? cO : cE;
      bl0 = (g & 1) ? dO : dE;
      bl1 = (g & 1) ? eO : eE;
    } else {
      const float p0 = v0 ? pr[j][0][0] * sv0 : 0.0f, p1 = v1 ? pr[j][0][1] * sv1 : 0.0f;
      uint32_t xh, xl;
      split_hi_lo(p0, p1, xh, xl);
      // Column g = 2q + part holds query q's hi (part 0) or lo (part 1) part.
      const uint32_t aH = __shfl_sync(kFull, xh, srcA), aL = __shfl_sync(kFull, xl, srcA);
      const uint32_t cH = __shfl_sync(kFull, xh, srcB), cL = __shfl_sync(kFull, xl, srcB);
      bh0 = (g & 1) ? aL : aH;
      bh1 = (g & 1) ? cL : cH;
      if ((g >> 1) >= G) bh0 = bh1 = 0u;
    }
    // V rows of tokens c, c+4, c+8, c+12; this thread's channels [16g, 16g+16).
    const uint2 t0 = *reinterpret_cast<const uint2*>(vb + (c + 0) * 64 + 8 * g);
    const uint2 t1 = *reinterpret_cast<const uint2*>(vb + (c + 4) * 64 + 8 * g);
    const uint2 t2 = *reinterpret_cast<const uint2*>(vb + (c + 8) * 64 + 8 * g);
    const uint2 t3 = *reinterpret_cast<const uint2*>(vb + (c + 12) * 64 + 8 * g);
    const uint32_t w0[2] = {t0.x, t0.y}, w1[2] = {t1.x, t1.y};
    const uint32_t w2[2] = {t2.x, t2.y}, w3[2] = {t3.x, t3.y};
#pragma unroll
    for (int i = 0; i < 8; i++) {  // m-tile i: byte i of the chunk = channels 16g+2i, +1
      const uint32_t e = i & 3;
      const uint32_t sel = e | (e << 4) | ((4 + e) << 8) | ((4 + e) << 12);
      const uint32_t r01 = prmt(w0[i >> 2], w1[i >> 2], sel);
      const uint32_t r23 = prmt(w2[i >> 2], w3[i >> 2], sel);
      const uint32_t a0 = nib_lo_to_half2(r01), a1 = nib_hi_to_half2(r01);
      const uint32_t a2 = nib_lo_to_half2(r23), a3 = nib_hi_to_half2(r23);
      mma_16816(st.o[i], a0, a1, a2, a3, bh0, bh1);
      if (G == 8) mma_16816(st.o[i], a0, a1, a2, a3, bl0, bl1);
    }
  }
}

// Bytes 0 and 2 of w, each two E2M1 codes (low nibble first) -> 2 x fp16x2, exact.
__device__ __forceinline__ void e2m1x2_b02_to_f16x2(uint32_t w, uint32_t& d0, uint32_t& d2) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b2;\n\t}"
      : "=r"(d0), "=r"(d2)
      : "r"(w));
}

// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t bitsel(uint32_t a, uint32_t b, uint32_t m) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(a), "r"(b), "r"(m));
  return r;
}

// PV of an NVFP4 tile with probabilities pr: as tile_pv, with P' = p; the V scales are
// applied in the dequantised A operand (the lane's channels 16g..16g+15 are block g of
// each token row, so a register's two tokens each take their own scale).
template <int G, int SEFF, typename N>
__device__ __forceinline__ void tile_pv4(State<G>& st, const uint8_t* slot, N ntok, int lane,
                                         const float (&pr)[2][QFrag4<G>::NQ][2]) {
  constexpr int RB = row_bytes(true);
  const int g = lane >> 2, c = lane & 3;
  const int tau0 = (g < 4) ? g : g + 4;
  const int tau1 = tau0 + 4;
  const int srcA = 4 * c + (g >> 1);
  const int srcB = srcA + 16;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const uint8_t* pbase = slot + (16 * j / SEFF) * (SEFF * RB);
    const int sl = (16 * j) % SEFF;
    const uint8_t* vb = pbase + SEFF * 64 + sl * 64;
    const uint8_t* vs = pbase + SEFF * 128 + SEFF * 8 + sl * 8;  // V scales [token][8]
    const bool v0 = tok_valid(ntok, j, tau0), v1 = tok_valid(ntok, j, tau1);
    uint32_t bh0, bh1, bl0 = 0u, bl1 = 0u;
    if (G == 8) {
      uint32_t xh[2], xl[2];
#pragma unroll
      for (int qq = 0; qq < 2; qq++) {
        const float p0 = v0 ? pr[j][qq][0] : 0.0f, p1 = v1 ? pr[j][qq][1] : 0.0f;
        split_hi_lo(p0, p1, xh[qq], xl[qq]);
      }
      const uint32_t aE = __shfl_sync(kFull, xh[0], srcA), aO = __shfl_sync(kFull, xh[1], srcA);
      const uint32_t cE = __shfl_sync(kFull, xh[0], srcB), cO = __shfl_sync(kFull, xh[1], srcB);
      const uint32_t dE = __shfl_sync(kFull, xl[0], srcA), dO = __shfl_sync(kFull, xl[1], srcA);
      const uint32_t eE = __shfl_sync(kFull, xl[0], srcB), eO = __shfl_sync(kFull, xl[1], srcB);
      bh0 = (g & 1) ? aO : aE;
      bh1 = (g & 1) ? cO : cE;
      bl0 = (g & 1) ? dO : dE;
      bl1 = (g & 1) ? eO : eE;
    } else {
      const float p0 = v0 ? pr[j][0][0] : 0.0f, p1 = v1 ? pr[j][0][1] : 0.0f;
      uint32_t xh, xl;
      split_hi_lo(p0, p1, xh, xl);
      const uint32_t aH = __shfl_sync(kFull, xh, srcA), aL = __shfl_sync(kFull, xl, srcA);
      const uint32_t cH = __shfl_sync(kFull, xh, srcB), cL = __shfl_sync(kFull, xl, srcB);
      bh0 = (g & 1) ? aL : aH;
      bh1 = (g & 1) ? cL : cH;
      if ((g >> 1) >= G) bh0 = bh1 = 0u;
    }
    // V rows of tokens c, c+4, c+8, c+12; this thread's channels [16g, 16g+16) = block g.
    const uint2 t0 = *reinterpret_cast<const uint2*>(vb + (c + 0) * 64 + 8 * g);
    const uint2 t1 = *reinterpret_cast<const uint2*>(vb + (c + 4) * 64 + 8 * g);
    const uint2 t2 = *reinterpret_cast<const uint2*>(vb + (c + 8) * 64 + 8 * g);
    const uint2 t3 = *reinterpret_cast<const uint2*>(vb + (c + 12) * 64 + 8 * g);
    // Tokens past the sequence's end take scale 0: their slot bytes are whatever the pool or
    // an earlier tile left there, and an E4M3 NaN would survive the zero probability.
    const uint32_t s0 = tok_valid(ntok, j, c) ? vs[(c + 0) * 8 + g] : 0u, s1 = tok_valid(ntok, j, c + 4) ? vs[(c + 4) * 8 + g] : 0u;
    const uint32_t s2 = tok_valid(ntok, j, c + 8) ? vs[(c + 8) * 8 + g] : 0u, s3 = tok_valid(ntok, j, c + 12) ? vs[(c + 12) * 8 + g] : 0u;
    const uint32_t s01 = s0 | (s1 << 8), s23 = s2 | (s3 << 8);
    const uint32_t S01 = e4m3x2_to_f16x2(s01), S23 = e4m3x2_to_f16x2(s23);
    const uint32_t w0[2] = {t0.x, t0.y}, w1[2] = {t1.x, t1.y};
    const uint32_t w2[2] = {t2.x, t2.y}, w3[2] = {t3.x, t3.y};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {  // m-tiles i, i + 1: bytes e, e + 1 of word i / 4
      const uint32_t e = i & 3;
      // bytes: [row0 byte e, row1 byte e, row0 byte e+1, row1 byte e+1]
      const uint32_t sel = e | ((4 + e) << 4) | ((e + 1) << 8) | ((5 + e) << 12);
      const uint32_t X01 = prmt(w0[i >> 2], w1[i >> 2], sel);
      const uint32_t X23 = prmt(w2[i >> 2], w3[i >> 2], sel);
      // even channels: low nibbles of the two tokens; odd: high nibbles (bytes 0 and 2)
      const uint32_t ev01 = bitsel(X01, X01 >> 4, 0x000F000Fu), od01 = bitsel(X01 >> 4, X01 >> 8, 0x000F000Fu);
      const uint32_t ev23 = bitsel(X23, X23 >> 4, 0x000F000Fu), od23 = bitsel(X23 >> 4, X23 >> 8, 0x000F000Fu);
      uint32_t a0[2], a1[2], a2[2], a3[2];
      e2m1x2_b02_to_f16x2(ev01, a0[0], a0[1]);
      e2m1x2_b02_to_f16x2(od01, a1[0], a1[1]);
      e2m1x2_b02_to_f16x2(ev23, a2[0], a2[1]);
      e2m1x2_b02_to_f16x2(od23, a3[0], a3[1]);
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const uint32_t A0 = hmul2(a0[h], S01), A1 = hmul2(a1[h], S01);
        const uint32_t A2 = hmul2(a2[h], S23), A3 = hmul2(a3[h], S23);
        mma_16816(st.o[i + h], A0, A1, A2, A3, bh0, bh1);
        if (G == 8) mma_16816(st.o[i + h], A0, A1, A2, A3, bl0, bl1);
      }
    }
  }
}

// Warp partial of one unit (its owned queries) -> a record block [G][kPartStride] at rec
// (shared or global memory): o'[128], m, l per query.  With qsel >= 0 only query qsel is
// written, at rec itself.
template <int G>
__device__ __forceinline__ void state_write(const State<G>& st, float* rec, int lane, int qsel = -1) {
  constexpr int NQ = State<G>::NQ;
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int qq = 0; qq < NQ; qq++) {
    float l = st.l[qq];
    l += __shfl_xor_sync(kFull, l, 4);
    l += __shfl_xor_sync(kFull, l, 8);
    l += __shfl_xor_sync(kFull, l, 16);
    const int qi = (G == 8) ? 2 * c + qq : c;
    if (qi >= G || (qsel >= 0 && qi != qsel)) continue;
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      if (G == 8) {
        v[2 * i] = st.o[i][qq];
        v[2 * i + 1] = st.o[i][2 + qq];
      } else {  // hi + lo columns
        v[2 * i] = st.o[i][0] + st.o[i][1];
        v[2 * i + 1] = st.o[i][2] + st.o[i][3];
      }
    }
    float* r = rec + (qsel >= 0 ? 0 : qi * kPartStride);
    float4* dst = reinterpret_cast<float4*>(r + 16 * g);
#pragma unroll
    for (int e = 0; e < 4; e++) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
    if (g == 0) {
      r[kD] = st.m[qq];
      r[kD + 1] = l;
    }
  }
}

// o'/l of one query (lane: channels 4*lane..4*lane+3) -> inverse block-diagonal
// Hadamard -> fp16 store.
__device__ __forceinline__ void finish_query(const float (&o)[4], float l, __half* dst, int lane,
                                             const DecodeParams& p) {
  float x[4];
  const float rl = l == 0.0f ? 0.0f : __frcp_rn(l);  // nothing attended: zeros
#pragma unroll
  for (int e = 0; e < 4; e++) x[e] = o[e] * rl;
  const int block = p.hadamard_block;
  {
    const bool rot = block > 1;  // b = 1 (plain INT4): no rotation
    const float a0 = x[0] + x[1], a1 = x[0] - x[1], a2 = x[2] + x[3], a3 = x[2] - x[3];
    x[0] = rot ? a0 + a2 : x[0];
    x[1] = rot ? a1 + a3 : x[1];
    x[2] = rot ? a0 - a2 : x[2];
    x[3] = rot ? a1 - a3 : x[3];
  }
#pragma unroll
  for (int s = 0; s < 5; s++) {
    if ((4 << s) < block) {
      const int bit = 1 << s;
      const float sgn = (lane & bit) ? -1.0f : 1.0f;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const float other = __shfl_xor_sync(kFull, x[e], bit);
        x[e] = __fmaf_rn(x[e], sgn, other);
      }
    }
  }
  const uint32_t lo = pack_half2(__float2half_rn(x[0] * p.cb), __float2half_rn(x[1] * p.cb));
  const uint32_t hi = pack_half2(__float2half_rn(x[2] * p.cb), __float2half_rn(x[3] * p.cb));
  *reinterpret_cast<uint2*>(dst + 4 * lane) = make_uint2(lo, hi);
}

// A unit with a single contributing warp (one tile): finish it from the warp's registers,
// one query at a time through a staging area of kPartStride floats.
template <int G>
__device__ __forceinline__ void finish_from_state(const State<G>& st, float* stage, __half* orow,
                                                  int lane, const DecodeParams& p) {
#pragma unroll 1
  for (int qi = 0; qi < G; qi++) {
    __syncwarp();
    state_write<G>(st, stage, lane, qi);
    __syncwarp();
    const float4 v = *reinterpret_cast<const float4*>(stage + 4 * lane);
    const float o[4] = {v.x, v.y, v.z, v.w};
    finish_query(o, stage[kD + 1], orow + qi * kD, lane, p);
  }
  __syncwarp();
}

template <bool GLOBAL>
__device__ __forceinline__ float2 ld_rec2(const float* a) {
  if (GLOBAL) return __ldcg(reinterpret_cast<const float2*>(a));
  return *reinterpret_cast<const float2*>(a);
}
template <bool GLOBAL>
__device__ __forceinline__ float4 ld_rec4(const float* a) {
  if (GLOBAL) return __ldcg(reinterpret_cast<const float4*>(a));
  return *reinterpret_cast<const float4*>(a);
}

// Merge of at most RMAX records (the common case: a unit's CTAs or a CTA's warps): every
// lane loads the (m, l) pairs and its o' slice of all records for two of the warp's queries
// at once (the (m, l) loads are broadcasts), so two queries cost one round trip and no
// cross-lane reduction.  Same contract as merge_records below.
template <int G, int QSTEP, bool GLOBAL, int RMAX, typename F>
__device__ __forceinline__ void merge_few(int nrec, F&& rec, int q0, __half* orow, float* crec,
                                          int lane, const DecodeParams& p) {
  constexpr int NQW = (G + QSTEP - 1) / QSTEP;  // queries this warp handles (at most)
  constexpr int QB = NQW < 2 ? NQW : 2;          // queries per round trip
#pragma unroll 1
  for (int qb = q0; qb < G; qb += QB * QSTEP) {
    float2 ml[QB][RMAX];
    float4 v[QB][RMAX];
#pragma unroll
    for (int i = 0; i < QB; i++) {
      const int qi = qb + i * QSTEP;
#pragma unroll
      for (int r = 0; r < RMAX; r++) {
        ml[i][r] = make_float2(-CUDART_INF_F, 0.0f);
        v[i][r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < nrec && qi < G) {
          const float* rr = rec(r) + qi * kPartStride;
          ml[i][r] = ld_rec2<GLOBAL>(rr + kD);
          v[i][r] = ld_rec4<GLOBAL>(rr + 4 * lane);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < QB; i++) {
      const int qi = qb + i * QSTEP;
      if (qi >= G) continue;
      float M = ml[i][0].x;
#pragma unroll
      for (int r = 1; r < RMAX; r++) M = fmaxf(M, ml[i][r].x);
      float o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, l = 0.0f;
#pragma unroll
      for (int r = 0; r < RMAX; r++) {
        const float e = (ml[i][r].x == -CUDART_INF_F) ? 0.0f : ex2_approx(ml[i][r].x - M);
        l += e * ml[i][r].y;
        o[0] += e * v[i][r].x;
        o[1] += e * v[i][r].y;
        o[2] += e * v[i][r].z;
        o[3] += e * v[i][r].w;
      }
      if (crec) {
        float* r = crec + qi * kPartStride;
        *reinterpret_cast<float4*>(r + 4 * lane) = make_float4(o[0], o[1], o[2], o[3]);
        if (lane == 0) *reinterpret_cast<float2*>(r + kD) = make_float2(M, l);
      } else {
        finish_query(o, l, orow + qi * kD, lane, p);
      }
    }
  }
}

// Per-warp fragment table: G queries x 96 words, at least one staging record.
// (NVFP4: G queries x 2 fp16 parts x 128 channels = G x 128 words.)
constexpr int frag_words(int g, bool fp4) {
  return (fp4 ? g * 128 : g * 96) > kPartStride ? (fp4 ? g * 128 : g * 96) : kPartStride;
}

// The format's q preparation, fragments and tile steps.
template <int G, int QSTEP, bool FP4>
__device__ __forceinline__ void prep_q(const uint8_t* qraw, uint32_t* frag, float* sf, int lane,
                                       const DecodeParams& p, int q0 = 0) {
  if constexpr (FP4) prep_q4_warp<G, QSTEP>(qraw, frag, sf, lane, p, q0);
  else prep_q_warp<G, QSTEP>(qraw, frag, sf, lane, p, q0);
}

template <int G, bool FP4>
struct QF {
  using type = QFrag<G>;
};
template <int G>
struct QF<G, true> {
  using type = QFrag4<G>;
};

template <int G>
__device__ __forceinline__ void qfrag_get(QFrag<G>& f, const uint32_t* qfb, const float* sfb, int lane) {
  qfrag_load<G>(f, qfb, sfb, lane);
}
template <int G>
__device__ __forceinline__ void qfrag_get(QFrag4<G>& f, const uint32_t* qfb, const float* sfb, int lane) {
  qfrag4_load<G>(f, qfb, sfb, lane);
}

template <int G, int SEFF, typename N>
__device__ __forceinline__ void tile_qk_any(const QFrag<G>& qf, const uint8_t* slot, N ntok, int lane,
                                            float (&sc)[2][QFrag<G>::NQ][2]) {
  tile_qk<G, SEFF>(qf, slot, ntok, lane, sc);
}
template <int G, int SEFF, typename N>
__device__ __forceinline__ void tile_qk_any(const QFrag4<G>& qf, const uint8_t* slot, N ntok, int lane,
                                            float (&sc)[2][QFrag4<G>::NQ][2]) {
  tile_qk4<G, SEFF>(qf, slot, ntok, lane, sc);
}

template <int G, int SEFF, bool FP4, typename N>
__device__ __forceinline__ void tile_pv_any(State<G>& st, const uint8_t* slot, N ntok, int lane,
                                            const float (&pr)[2][QFrag<G>::NQ][2]) {
  if constexpr (FP4) tile_pv4<G, SEFF>(st, slot, ntok, lane, pr);
  else tile_pv<G, SEFF>(st, slot, ntok, lane, pr);
}

}  // namespace

}  // namespace kvq
