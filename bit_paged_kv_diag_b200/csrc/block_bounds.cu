// block_bounds.cu -- per-page bounds of the cached keys, for sm_100a.
//
// Mathematics.  For every page of an append's tokens and every KV head, over the page's filled
// slots: mx_d and mn_d, the largest and smallest of channel d of the cached (rotated) keys s * n,
// exact in fp32 (an fp16 scale of 11 bits times a 4-bit integer; E2M1 times E4M3 is exact in
// fp16).  With a = max_d max(|mx_d|, |mn_d|), sigma is the least power of two with 127 sigma >= a
// (0 when a = 0) and hi_d = ceil(mx_d / sigma), lo_d = floor(mn_d / sigma) are int8: outward, so
// that lo_d sigma <= k_d <= hi_d sigma holds for every key of the page and a score from the
// bounds is never below a key's own.  A power of two keeps both divisions exact.
//
// Layout.  One warp per (page, head), lane j the channels 4j .. 4j + 3: a row is one 64-byte
// load of the warp, no lane ever exchanges channels, and the only reduction is that of a.  Rows
// go in pairs, so that each nibble expansion yields one channel of two rows and the running
// bounds take three-operand minima and maxima.
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include "append_row.cuh"
#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

namespace {

constexpr int kD = 128;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 16;  // rows in flight per warp

__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ uint32_t h2min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t h2max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// n * s in fp32 of two fp16 values, exact (22 bits).
__device__ __forceinline__ float mul_f16(uint32_t n, uint32_t s) {
  float d;
  asm("fma.rn.f32.f16 %0, %1, %2, %3;"
      : "=f"(d)
      : "h"(static_cast<uint16_t>(n)), "h"(static_cast<uint16_t>(s)), "f"(-0.0f));
  return d;
}

template <bool FP4>
__global__ void __launch_bounds__(kThreads) bounds_kernel(BoundsParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int gw = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int item = gw / p.num_kv_heads, h = gw - item * p.num_kv_heads;
  // Item slots: sequence b has those from cu[b] / S + 2 b on, at least as many as the pages that
  // its tokens can touch ((n - 1) / S + 2), so an item finds its sequence without a prefix sum.
  auto slot0 = [&](int b) { return (__ldg(p.cu_new_tokens + b) >> p.page_shift) + 2 * b; };
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (slot0(mid) <= item) lo = mid; else hi = mid;
  }
  const int n = __ldg(p.cu_new_tokens + lo + 1) - __ldg(p.cu_new_tokens + lo);
  const int j = item - slot0(lo);
  if (n <= 0 || j < 0) return;
  const int S = p.page_size, before = __ldg(p.seq_lens + lo);
  const long long cap = static_cast<long long>(p.max_pages_per_seq) << p.page_shift;
  const long long after = static_cast<long long>(before) + n;
  if (before < 0 || after > cap) {
    if (j == 0 && lane == 0) atomicOr(p.status, KVQ_DEV_BAD_POS_BIT);
    if (before < 0) return;
  }
  const long long lp = (before >> p.page_shift) + static_cast<long long>(j);
  const long long left = (after < cap ? after : cap) - (lp << p.page_shift);
  if (left <= 0) return;
  const int filled = left < S ? static_cast<int>(left) : S;
  const int page = __ldg(p.page_table + static_cast<size_t>(lo) * p.max_pages_per_seq + lp);
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) atomicOr(p.status, KVQ_DEV_BAD_PAGE_BIT);
    return;
  }
  constexpr int kScaleBytes = FP4 ? kD / 16 : 2;
  const uint8_t* blk = p.pool_layer + (static_cast<size_t>(page) * p.num_kv_heads + h) *
                                          (static_cast<size_t>(S) * (kD + 2 * kScaleBytes));
  const unsigned short* codes = reinterpret_cast<const unsigned short*>(blk) + lane;
  const uint8_t* scales = blk + S * kD;

  float mx[4], mn[4];
  uint32_t hx[4], hn[4];  // NVFP4: the same of even and odd rows, as fp16 pairs
#pragma unroll
  for (int e = 0; e < 4; e++) {
    mx[e] = -CUDART_INF_F;
    mn[e] = CUDART_INF_F;
    hx[e] = 0xFC00FC00u;
    hn[e] = 0x7C007C00u;
  }
  for (int r0 = 0; r0 < filled; r0 += kChunk) {
    uint32_t c[kChunk], s[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; i++) {
      const int r = min(r0 + i, filled - 1);  // rows past the end repeat the last one
      c[i] = __ldcg(codes + r * (kD / 4));
      if constexpr (FP4) s[i] = __ldcg(scales + r * kScaleBytes + (lane >> 2));
      else s[i] = __ldcg(reinterpret_cast<const unsigned short*>(scales) + r);
    }
#pragma unroll
    for (int i = 0; i < kChunk; i += 2) {
      if constexpr (FP4) {
        uint32_t sh;  // E4M3 -> fp16, exact: both rows' scales
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sh) : "h"(static_cast<uint16_t>(s[i] | (s[i + 1] << 8))));
        // Row i's and row i + 1's channels as fp16 pairs (channel 2e, 2e + 1).
        const uint32_t w = prmt(c[i], c[i + 1], 0x5410u);
        uint32_t v[4];
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
            : "r"(w));
        const uint32_t S0 = prmt(sh, sh, 0x1010u), S1 = prmt(sh, sh, 0x3232u);
#pragma unroll
        for (int e = 0; e < 4; e++) {
          uint32_t x;
          asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(v[e]), "r"(e < 2 ? S0 : S1));
          hx[e] = h2max(hx[e], x);
          hn[e] = h2min(hn[e], x);
        }
      } else {
        const uint32_t w = prmt(c[i], c[i + 1], 0x5410u);  // row i low, row i + 1 high
        const uint32_t v[4] = {nib_lo_to_half2(w), nib_hi_to_half2(w), nib_lo_to_half2(w >> 8),
                               nib_hi_to_half2(w >> 8)};
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float a = mul_f16(v[e] & 0xFFFFu, s[i]), b = mul_f16(v[e] >> 16, s[i + 1]);
          mx[e] = max3(mx[e], a, b);
          mn[e] = min3(mn[e], a, b);
        }
      }
    }
  }
  if constexpr (FP4) {
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const uint32_t x = h2max(hx[e], hx[e + 2]), y = h2min(hn[e], hn[e + 2]);
      mx[2 * e] = cvt_f16(x & 0xFFFFu);
      mx[2 * e + 1] = cvt_f16(x >> 16);
      mn[2 * e] = cvt_f16(y & 0xFFFFu);
      mn[2 * e + 1] = cvt_f16(y >> 16);
    }
  }
  float a = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; e++) a = max3(a, fabsf(mx[e]), fabsf(mn[e]));
#pragma unroll
  for (int d = 1; d < 32; d *= 2) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
  // 127 / 64 has the mantissa 0x7E0000: a <= 127 * 2^k with k = exponent(a) - 6, or one more.
  const uint32_t bits = __float_as_uint(a);
  const int ef = static_cast<int>(bits >> 23) - 6 + ((bits & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  const float sigma = a > 0.0f && ef > 0 ? __uint_as_float(static_cast<uint32_t>(ef) << 23) : 0.0f;
  const float inv = sigma > 0.0f ? __uint_as_float(static_cast<uint32_t>(254 - ef) << 23) : 0.0f;
  uint32_t wl = 0, wh = 0;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const int cl = static_cast<int>(fmaxf(floorf(mn[e] * inv), -127.0f));
    const int ch = static_cast<int>(fminf(ceilf(mx[e] * inv), 127.0f));
    wl |= (static_cast<uint32_t>(cl) & 0xFFu) << (8 * e);
    wh |= (static_cast<uint32_t>(ch) & 0xFFu) << (8 * e);
  }
  const size_t row = static_cast<size_t>(page) * p.num_kv_heads + h;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.codes + row * (2 * kD));
  dst[lane] = wl;
  dst[32 + lane] = wh;
  if (lane == 0) p.scale[row] = sigma;
}

}  // namespace

int launch_bounds(const BoundsParams& p, bool fp4, cudaStream_t stream) {
  if (p.total_new_tokens == 0) return 0;
  const long long items = (static_cast<long long>(p.total_new_tokens) >> p.page_shift) + 2LL * p.batch;
  const long long warps = items * p.num_kv_heads;
  if (warps > 0x7fffffffLL - kWarps) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (fp4 ? cudaLaunchKernelEx(&cfg, bounds_kernel<true>, p) : cudaLaunchKernelEx(&cfg, bounds_kernel<false>, p)) ==
                 cudaSuccess
             ? 0
             : -2;
}

}  // namespace kvq
