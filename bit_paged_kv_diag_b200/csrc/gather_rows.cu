// gather_rows.cu -- cached K and V rows read back in the model's basis, for sm_100a.
//
// Mathematics.  A row is y = s * n (INT4: n the 4-bit integers, s the row's fp16 scale; NVFP4:
// n the E2M1 values, s the E4M3 scale of each 16 channels), rotated back by the cache's
// block-diagonal Hadamard transform, x = c_b * (butterfly of y) -- the orthonormal Sylvester
// matrix is its own inverse -- and rounded once to fp16 or bf16.  INT4: the butterfly runs on
// the integers in fp16 pairs, where every sum is exact (|sum| <= 8 * 128 = 2^10), and s * c_b
// is applied afterwards in fp32 (two roundings of 2^-24 next to the output's 2^-11 or 2^-8).
// NVFP4: the stages inside a block of 16 channels are exact in fp16 as well (|sum| <= 6 * 16
// in steps of 1/2); the scales and the stages across blocks are fp32.
//
// Layout.  A warp takes the K and the V rows of 16 consecutive tokens of one KV head (1 KB of
// codes each, contiguous inside a page, all in flight at once); two lanes hold a row, lane l the channels [64 l, 64 l + 64),
// so that only b = 128 exchanges data between lanes.  The finished rows go through shared memory
// and leave by one bulk copy each: stored from registers, a lane's 128 bytes are a line of their
// own in every store and the L1 data path takes 32 passes per kilobyte.  Slot t of lane l holds
// the chunk (8 channels) t ^ 4 l, so that with rows 272 bytes apart the lanes' 16-byte stores hit
// all banks evenly; the stage h = 32 and the exchange of h = 64 account for that order.
//
// Measured, the kernel alone behind a flush of L2: 65,536 INT4 tokens x 8 heads (b = 128) 72 us, 4.7 TB/s; 161,700 NVFP4 tokens x 4 heads
// (b = 64) 84 us, 5.0 TB/s -- 0.72 and 0.77 of the copy rate.  The arithmetic pipe is busy for 57 %
// of the time, the issue slots for 65 %.  Stores straight from registers took 95 and 103 us, one of
// K and V per warp 86 and 90 us.
#include <cuda_fp16.h>
#include <stdint.h>

#include "append_row.cuh"
#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

namespace {

constexpr int kD = 128;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerWarp = 16;
constexpr int kRowStride = 2 * kD + 16;  // bytes between rows in shared memory

__device__ __forceinline__ uint32_t h2add(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t h2sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t h2fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// (a, c) -> (a + c, a - c) of registers i and i + step, for all pairs with bit `step` of i clear.
template <int N>
__device__ __forceinline__ void h2_stage(uint32_t (&x)[N], int step) {
#pragma unroll
  for (int i = 0; i < N; i++) {
    if (i & step) continue;
    const uint32_t a = x[i], c = x[i + step];
    x[i] = h2add(a, c);
    x[i + step] = h2sub(a, c);
  }
}

// The stage inside a register's pair: (lo, hi) -> (lo + hi, lo - hi).
template <int N>
__device__ __forceinline__ void h2_pair_stage(uint32_t (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i++) x[i] = h2fma(x[i], 0xBC003C00u, prmt(x[i], x[i], 0x1032u));  // (1, -1)
}

// Two fp32 values -> two fp16 or bf16 (lo -> low half), nearest even.
template <bool BF16>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 1-D bulk copy of this CTA's shared memory to global memory (16-byte aligned, whole 16-byte
// units), and the wait until the copies' reads of shared memory are done.
__device__ __forceinline__ void bulk_copy_s2g(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// The lane's 64 channels of an INT4 row: 8 words of codes (slot order) -> 32 words of outputs.
template <int BLOCK, bool BF16>
__device__ __forceinline__ void row_int4(const uint32_t (&w)[8], float f, int l, unsigned pmask, uint32_t (&o)[32]) {
  // x[4c + s] = channels 8c + s (low half) and 8c + s + 4 (high half)
  uint32_t x[32];
#pragma unroll
  for (int c = 0; c < 8; c++) {
    x[4 * c] = nib_lo_to_half2(w[c]);
    x[4 * c + 1] = nib_hi_to_half2(w[c]);
    x[4 * c + 2] = nib_lo_to_half2(w[c] >> 8);
    x[4 * c + 3] = nib_hi_to_half2(w[c] >> 8);
  }
  if constexpr (BLOCK > 1) {
    h2_stage(x, 1);
    h2_stage(x, 2);
    h2_pair_stage(x);
    h2_stage(x, 4);
    h2_stage(x, 8);
  }
  const uint32_t sg = l ? 0xBC00BC00u : 0x3C003C00u, nsg = l ? 0x3C003C00u : 0xBC00BC00u;
  if constexpr (BLOCK >= 64) {
    // h = 32: slots t and t + 4; in lane 1 slot t is the upper chunk.
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const uint32_t a = x[i], c = x[i + 16];
      x[i] = h2fma(a, sg, c);
      x[i + 16] = h2fma(c, nsg, a);
    }
  }
  if constexpr (BLOCK == 128) {
    // h = 64: lane 0 keeps own + other, lane 1 other - own; the partner of slot t is slot t ^ 4.
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const uint32_t ra = __shfl_xor_sync(pmask, x[i + 16], 1), rc = __shfl_xor_sync(pmask, x[i], 1);
      x[i] = h2fma(x[i], sg, ra);
      x[i + 16] = h2fma(x[i + 16], sg, rc);
    }
  }
#pragma unroll
  for (int c = 0; c < 8; c++) {
    float v[8];
#pragma unroll
    for (int s = 0; s < 4; s++) {
      v[s] = __fmul_rn(cvt_f16(x[4 * c + s] & 0xFFFFu), f);
      v[s + 4] = __fmul_rn(cvt_f16(x[4 * c + s] >> 16), f);
    }
#pragma unroll
    for (int e = 0; e < 4; e++) o[4 * c + e] = narrow<BF16>(v[2 * e], v[2 * e + 1]);
  }
}

// The same of an NVFP4 row; sc = the lane's 4 E4M3 scale bytes in slot order.
template <int BLOCK, bool BF16>
__device__ __forceinline__ void row_fp4(const uint32_t (&w)[8], uint32_t sc, float cb, int l, unsigned pmask,
                                        uint32_t (&o)[32]) {
  f2 y[32];  // channels 2i, 2i + 1
  const float2 s01 = e4m3x2_value(sc & 0xFFFFu), s23 = e4m3x2_value(sc >> 16);
  const float sv[4] = {s01.x, s01.y, s23.x, s23.y};
#pragma unroll
  for (int b = 0; b < 4; b++) {
    uint32_t x[8];
#pragma unroll
    for (int j = 0; j < 2; j++)
      asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
          "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
          : "=r"(x[4 * j]), "=r"(x[4 * j + 1]), "=r"(x[4 * j + 2]), "=r"(x[4 * j + 3])
          : "r"(w[2 * b + j]));
    if constexpr (BLOCK > 1) {
      h2_pair_stage(x);
      h2_stage(x, 1);
      h2_stage(x, 2);
      h2_stage(x, 4);
    }
    const f2 S = pk(sv[b], sv[b]);
#pragma unroll
    for (int i = 0; i < 8; i++) y[8 * b + i] = mul2(pk(cvt_f16(x[i] & 0xFFFFu), cvt_f16(x[i] >> 16)), S);
  }
  if constexpr (BLOCK > 1) {
#pragma unroll
    for (int i = 0; i < 32; i++) {  // h = 16
      if (i & 8) continue;
      const f2 a = y[i], c = y[i + 8];
      y[i] = add2(a, c);
      y[i + 8] = sub2(a, c);
    }
  }
  const float sg = l ? -1.0f : 1.0f;
  const f2 SG = pk(sg, sg), NSG = pk(-sg, -sg);
  if constexpr (BLOCK >= 64) {
#pragma unroll
    for (int i = 0; i < 16; i++) {  // h = 32
      const f2 a = y[i], c = y[i + 16];
      y[i] = fma2(a, SG, c);
      y[i + 16] = fma2(c, NSG, a);
    }
  }
  if constexpr (BLOCK == 128) {
#pragma unroll
    for (int i = 0; i < 16; i++) {  // h = 64
      float a0, a1, c0, c1;
      upk(y[i], a0, a1);
      upk(y[i + 16], c0, c1);
      const f2 ra = pk(__shfl_xor_sync(pmask, c0, 1), __shfl_xor_sync(pmask, c1, 1));
      const f2 rc = pk(__shfl_xor_sync(pmask, a0, 1), __shfl_xor_sync(pmask, a1, 1));
      y[i] = fma2(y[i], SG, ra);
      y[i + 16] = fma2(y[i + 16], SG, rc);
    }
  }
  const f2 CB = pk(cb, cb);
#pragma unroll
  for (int i = 0; i < 32; i++) {
    float a, c;
    upk(BLOCK > 1 ? mul2(y[i], CB) : y[i], a, c);
    o[i] = narrow<BF16>(a, c);
  }
}

template <int BLOCK, bool FP4, bool BF16>
__global__ void __launch_bounds__(kThreads, 4) gather_kernel(GatherParams p) {
  __shared__ __align__(128) uint8_t stage[kWarps][2][kRowsPerWarp * kRowStride];
  // (No early launch of the next kernel, whose blocks would take the room of this one's: an append and
  // a read-back of 16 tokens in turn, 9.3 us a pair; with it 9.7.)
  griddep_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, l = lane & 1;
  const unsigned pmask = 0x3u << (lane & 30);
  // Item: (16 tokens, head), the head fastest.
  const int item = blockIdx.x * kWarps + w;
  const int tg = item / p.num_kv_heads, h = item - tg * p.num_kv_heads;
  const int t = tg * kRowsPerWarp + (lane >> 1);
  int first, next;
  const SeqWindow win = seq_window(p.cu_rows, p.batch, tg * kRowsPerWarp);
  const int lo = seq_find(win, p.cu_rows, p.batch, t, first, next);
  bool have = t < p.total_rows;  // (the same in both lanes of a row)
  if (have) {
    have = t >= first && t < next;  // otherwise a row of no sequence: left as it is
    if (have) {
      const long long pos = static_cast<long long>(__ldg(p.starts + lo)) + (t - first);
      int page = -1;
      const bool bad_pos = pos < 0 || (pos >> p.page_shift) >= p.max_pages_per_seq;
      if (!bad_pos) page = __ldg(p.page_table + static_cast<size_t>(lo) * p.max_pages_per_seq + (pos >> p.page_shift));
      const bool good = page >= 0 && page < p.num_pages;
      if (!good) atomicOr(p.status, bad_pos ? KVQ_DEV_BAD_POS_BIT : KVQ_DEV_BAD_PAGE_BIT);
      // Both rows' codes and scales (zeros for a bad page), in flight together.
      constexpr int kScaleBytes = FP4 ? kD / 16 : 2;
      uint4 ca[2], cb[2];
      uint32_t sb[2] = {0u, 0u};
#pragma unroll
      for (int kv = 0; kv < 2; kv++) ca[kv] = cb[kv] = make_uint4(0u, 0u, 0u, 0u);
      if (good) {
        const int S = p.page_size, slot = static_cast<int>(pos) & (S - 1);
        const uint8_t* blk = p.pool_layer + (static_cast<size_t>(page) * p.num_kv_heads + h) *
                                                (static_cast<size_t>(S) * (kD + 2 * kScaleBytes));
#pragma unroll
        for (int kv = 0; kv < 2; kv++) {
          if (!(kv ? p.v_out : p.k_out)) continue;
          const uint4* src = reinterpret_cast<const uint4*>(blk + (kv * S + slot) * (kD / 2) + 32 * l);
          const uint8_t* sp = blk + S * kD + (kv * S + slot) * kScaleBytes;
          ca[kv] = __ldcg(src + l);  // slot t = chunk t ^ 4 l
          cb[kv] = __ldcg(src + (l ^ 1));
          if constexpr (FP4) sb[kv] = __ldcg(reinterpret_cast<const uint32_t*>(sp) + l);
          else sb[kv] = __ldcg(reinterpret_cast<const unsigned short*>(sp));
        }
      }
#pragma unroll
      for (int kv = 0; kv < 2; kv++) {
        if (!(kv ? p.v_out : p.k_out)) continue;
        const uint32_t cw[8] = {ca[kv].x, ca[kv].y, ca[kv].z, ca[kv].w, cb[kv].x, cb[kv].y, cb[kv].z, cb[kv].w};
        uint32_t o[32];
        if constexpr (FP4) {
          row_fp4<BLOCK, BF16>(cw, l ? prmt(sb[kv], sb[kv], 0x1032u) : sb[kv], p.cb, l, pmask, o);
        } else {
          const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(sb[kv])));
          row_int4<BLOCK, BF16>(cw, BLOCK > 1 ? __fmul_rn(s, p.cb) : s, l, pmask, o);
        }
        const uint32_t dst = smem_addr(stage[w][kv]) + (lane >> 1) * kRowStride + 128 * l;
#pragma unroll
        for (int i = 0; i < 8; i++)
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst + 16 * (i ^ (4 * l))), "r"(o[4 * i]),
                       "r"(o[4 * i + 1]), "r"(o[4 * i + 2]), "r"(o[4 * i + 3])
                       : "memory");
        // The row leaves when both of its lanes have stored.
        fence_proxy_async_smem();
        __syncwarp(pmask);
        if (l == 0) {
          uint8_t* const out = static_cast<uint8_t*>(kv ? p.v_out : p.k_out);
          bulk_copy_s2g(out + (static_cast<size_t>(t) * p.num_kv_heads + h) * (2 * kD),
                        smem_addr(stage[w][kv]) + (lane >> 1) * kRowStride, 2 * kD);
          bulk_commit();
        }
      }
    }
  }
  if (have && l == 0) bulk_wait_read();  // the copies read this CTA's memory: stay until they have
}

template <int BLOCK, bool FP4>
int launch_one(const cudaLaunchConfig_t& cfg, const GatherParams& p, bool bf16) {
  return (bf16 ? cudaLaunchKernelEx(&cfg, gather_kernel<BLOCK, FP4, true>, p)
               : cudaLaunchKernelEx(&cfg, gather_kernel<BLOCK, FP4, false>, p)) == cudaSuccess
             ? 0
             : -2;
}

template <bool FP4>
int launch_block(const cudaLaunchConfig_t& cfg, const GatherParams& p, int block, bool bf16) {
  switch (block) {
    case 1: return launch_one<1, FP4>(cfg, p, bf16);
    case 32: return launch_one<32, FP4>(cfg, p, bf16);
    case 64: return launch_one<64, FP4>(cfg, p, bf16);
    case 128: return launch_one<128, FP4>(cfg, p, bf16);
    default: return -1;
  }
}

}  // namespace

int launch_gather(const GatherParams& p, int block, bool fp4, bool bf16, cudaStream_t stream) {
  if (p.total_rows == 0) return 0;
  const long long items =
      (static_cast<long long>(p.total_rows) + kRowsPerWarp - 1) / kRowsPerWarp * p.num_kv_heads;
  if (items > 0x7fffffffLL - kWarps) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((items + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return fp4 ? launch_block<true>(cfg, p, block, bf16) : launch_block<false>(cfg, p, block, bf16);
}

}  // namespace kvq
