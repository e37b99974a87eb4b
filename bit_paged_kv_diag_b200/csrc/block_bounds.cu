// block_bounds.cu -- per-page bounds of the cached keys, for sm_100a.
//
// Mathematics.  For every page of an append's tokens and every KV head, over the page's filled
// slots: mx_d and mn_d, the largest and smallest of channel d of the cached (rotated) keys s * n,
// exact in fp32 (an fp16 scale of 11 bits times a 4-bit integer; E2M1 times E4M3 is exact in
// fp16).  With a = max_d max(|mx_d|, |mn_d|), sigma is the least power of two with 127 sigma >= a
// (0 when a = 0) and hi_d = ceil(mx_d / sigma), lo_d = floor(mn_d / sigma) are int8: outward, so
// that lo_d sigma <= k_d <= hi_d sigma holds for every key of the page and a score from the
// bounds is never below a key's own with the same query (which the page choice rounds to int8).  A power of two keeps both divisions exact.
//
// Layout.  One warp per (page, head); the page's key codes and scales come by bulk copies of up to
// 64 rows into the warp's own two shared-memory slots (loaded straight into registers, the
// compiler kept only a few rows in flight and the kernel waited on memory for most of its time).
// Half a warp takes a row, lane j of a half the channels 8j .. 8j + 7.  A half's rows go in pairs,
// so that each nibble expansion yields one channel of two rows and the running bounds take
// three-operand minima and maxima; the halves meet once at the end.
//
// Measured, the kernel alone behind a flush of L2: 8 x 8192 INT4 tokens in pages of 64, 8 heads: 19.5
// us for 38 MB (5.8 us at the copy rate); the arithmetic pipe (conversions, minima, maxima) is busy for 60 % of it.  The last pages
// of 256 sequences: 7.0 us, a chain of four memory round trips.
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
constexpr int kRows = 64;                         // rows of a slot
constexpr int kScaleMax = kD / 16;                // scale bytes of a row at most
constexpr int kStep = 8;                          // rows of a half in registers
constexpr int kSlot = kRows * (kD / 2 + kScaleMax);
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // bounded waits: 2 s

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
  __shared__ __align__(128) uint8_t ring[kWarps][2][kSlot];
  __shared__ __align__(8) uint64_t bars[kWarps][2];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint32_t bar = smem_addr(bars[w]);
  if (lane == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 8, 1);
    fence_mbar_init();
  }
  __syncwarp();
  griddep_wait();
  const int gw = blockIdx.x * kWarps + w;
  const int item = gw / p.num_kv_heads, h = gw - item * p.num_kv_heads;
  // Item slots: sequence b has those from cu[b] / S + 2 b on, at least as many as the pages that
  // its tokens can touch ((n - 1) / S + 2), so an item finds its sequence without a prefix sum.
  auto slot0 = [&](int b) { return (__ldg(p.cu_new_tokens + b) >> p.page_shift) + 2 * b; };
  const int lo = warp_find(p.batch, item, slot0);
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
  const int half = lane >> 4, j8 = lane & 15;
  // Rows [64 i, 64 i + 64) of the page, as far as they are filled (scales in whole 16 bytes).
  auto fetch = [&](int i) {
    const int n = min(kRows, filled - i * kRows);
    if (lane != 0 || n <= 0) return;
    const uint32_t dst = smem_addr(ring[w][i & 1]), b = bar + 8 * (i & 1);
    const uint32_t scale_bytes = (static_cast<uint32_t>(n) * kScaleBytes + 15) & ~15u;
    mbar_arrive_expect_tx(b, n * (kD / 2) + scale_bytes);
    bulk_copy_g2s(dst, blk + i * kRows * (kD / 2), n * (kD / 2), b, 0ull);
    bulk_copy_g2s(dst + kRows * (kD / 2), blk + S * kD + i * kRows * kScaleBytes, scale_bytes, b, 0ull);
  };
  fetch(0);
  fetch(1);

  float mx[8], mn[8];
  uint32_t hx[8], hn[8];  // NVFP4: of the pair's two rows, as fp16 pairs of channels 2e, 2e + 1
#pragma unroll
  for (int e = 0; e < 8; e++) {
    mx[e] = -CUDART_INF_F;
    mn[e] = CUDART_INF_F;
    hx[e] = 0xFC00FC00u;
    hn[e] = 0x7C007C00u;
  }
  for (int q = 0; q * kRows < filled; q++) {
    if (!mbar_wait_warp(bar + 8 * (q & 1), (q >> 1) & 1, kWaitLimitNs)) {
      // Flag it and let the copies in flight land (bounded) before their memory is reused.
      if (lane == 0) atomicOr(p.status, KVQ_DEV_TIMEOUT_BIT);
      mbar_wait_warp(bar + 8 * (q & 1), (q >> 1) & 1, kWaitLimitNs);
      if ((q + 1) * kRows < filled) mbar_wait_warp(bar + 8 * ((q + 1) & 1), ((q + 1) >> 1) & 1, kWaitLimitNs);
      return;
    }
    const uint8_t* slot = ring[w][q & 1];
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(slot) + j8;
    const uint8_t* scales = slot + kRows * (kD / 2);
    const int n = min(kRows, filled - q * kRows);
    for (int r0 = half; r0 < n + half; r0 += 2 * kStep) {
      uint32_t c[kStep], s[kStep];
#pragma unroll
      for (int i = 0; i < kStep; i++) {
        const int r = min(r0 + 2 * i, n - 1);  // rows past the end repeat the last one
        c[i] = codes[r * (kD / 8)];
        if constexpr (FP4) s[i] = scales[r * kScaleBytes + (j8 >> 1)];
        else s[i] = reinterpret_cast<const uint16_t*>(scales)[r];
      }
#pragma unroll
      for (int i = 0; i < kStep; i += 2) {
        if constexpr (FP4) {
          uint32_t sh;  // E4M3 -> fp16, exact: both rows' scales
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sh) : "h"(static_cast<uint16_t>(s[i] | (s[i + 1] << 8))));
#pragma unroll
          for (int z = 0; z < 2; z++) {
            const uint32_t f = prmt(sh, sh, z ? 0x3232u : 0x1010u);
            uint32_t v[4];  // channels 2e, 2e + 1
            asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
                "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
                "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
                : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                : "r"(c[i + z]));
#pragma unroll
            for (int e = 0; e < 4; e++) {
              uint32_t x;
              asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(v[e]), "r"(f));
              hx[4 * z + e] = h2max(hx[4 * z + e], x);
              hn[4 * z + e] = h2min(hn[4 * z + e], x);
            }
          }
        } else {
#pragma unroll
          for (int z = 0; z < 2; z++) {  // channels 4z .. 4z + 3
            const uint32_t w = prmt(c[i], c[i + 1], z ? 0x7632u : 0x5410u);  // one row low, the other high
            const uint32_t v[4] = {nib_lo_to_half2(w), nib_hi_to_half2(w), nib_lo_to_half2(w >> 8),
                                   nib_hi_to_half2(w >> 8)};
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const float x0 = mul_f16(v[e] & 0xFFFFu, s[i]), x1 = mul_f16(v[e] >> 16, s[i + 1]);
              mx[4 * z + e] = max3(mx[4 * z + e], x0, x1);
              mn[4 * z + e] = min3(mn[4 * z + e], x0, x1);
            }
          }
        }
      }
    }
    // The slot is read: it can take the rows after the next.
    __syncwarp();
    if ((q + 2) * kRows < filled) {
      fence_proxy_async_smem();
      fetch(q + 2);
    }
  }
  if constexpr (FP4) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const uint32_t x = h2max(hx[e], hx[e + 4]), y = h2min(hn[e], hn[e + 4]);
      mx[2 * e] = cvt_f16(x & 0xFFFFu);
      mx[2 * e + 1] = cvt_f16(x >> 16);
      mn[2 * e] = cvt_f16(y & 0xFFFFu);
      mn[2 * e + 1] = cvt_f16(y >> 16);
    }
  }
  // The halves meet: half 0 keeps the maxima, half 1 the minima.
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const float other = __shfl_xor_sync(0xffffffffu, half ? mx[e] : mn[e], 16);
    v[e] = half ? fminf(mn[e], other) : fmaxf(mx[e], other);
  }
  uint32_t ab = 0;  // (absolute values are ordered as their bits)
#pragma unroll
  for (int e = 0; e < 8; e++) ab = max(ab, __float_as_uint(fabsf(v[e])));
  const float a = __uint_as_float(__reduce_max_sync(0xffffffffu, ab));
  // 127 / 64 has the mantissa 0x7E0000: a <= 127 * 2^k with k = exponent(a) - 6, or one more.
  const uint32_t bits = __float_as_uint(a);
  const int ef = static_cast<int>(bits >> 23) - 6 + ((bits & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  const float sigma = a > 0.0f && ef > 0 ? __uint_as_float(static_cast<uint32_t>(ef) << 23) : 0.0f;
  const float inv = sigma > 0.0f ? __uint_as_float(static_cast<uint32_t>(254 - ef) << 23) : 0.0f;
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const float t = v[e] * inv;
    const int code = static_cast<int>(half ? fmaxf(floorf(t), -127.0f) : fminf(ceilf(t), 127.0f));
    out[e >> 2] |= (static_cast<uint32_t>(code) & 0xFFu) << (8 * (e & 3));
  }
  const size_t row = static_cast<size_t>(page) * p.num_kv_heads + h;
  reinterpret_cast<uint2*>(p.codes + row * (2 * kD) + (half ? 0 : kD))[j8] = make_uint2(out[0], out[1]);
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
  const cudaError_t rc =
      fp4 ? cudaLaunchKernelEx(&cfg, bounds_kernel<true>, p) : cudaLaunchKernelEx(&cfg, bounds_kernel<false>, p);
  return rc == cudaSuccess ? 0 : -2;
}

}  // namespace kvq
