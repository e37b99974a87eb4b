// rope_append.cu -- append of K and V to the paged 4-bit cache with the position rotation of
// q and k applied on the way, for sm_100a.
//
// Mathematics.  Token at position p, pair i of the rotary_dim / 2 rotated channel pairs:
// theta = p * inv_freq[i] in fp64, c = fl32(factor cos theta), s = fl32(factor sin theta), and
//   x'_a = fl(fl(x_a c) - fl(x_b s)),  x'_b = fl(fl(x_b c) + fl(x_a s))
// with (a, b) = (i, i + rotary_dim / 2), or (2i, 2i + 1) for the interleaved form.  The angle
// is formed in fp64 because an fp32 product of a far position loses the angle itself (2^17
// tokens times 1 leaves 2^-7 radian); every rounding above is fixed, so that the stored codes
// are those of any implementation that rounds the same way.  The rotated k stays in fp32 on its way into the block-diagonal Hadamard
// butterfly and the quantiser (append_row.cuh), which are the append kernel's; q' is rounded
// once to fp16, the type that the attention calls read.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>

#include "append_row.cuh"
#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

namespace {

constexpr int kD = 128;
constexpr int kRow = 2 * kD;          // bytes of one fp16 / bf16 row
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kStageRows = 16;        // rows of a warp stage: two lanes per row
constexpr int kTileRows = 192;        // rows of a CTA's tile, about 48 KB
constexpr int kRopeTokens = 32;       // tokens of a tile at most
constexpr int kMaxSmem = (kTileRows + 3 * 15) * kRow + kRopeTokens * (kD * 4 + 16) + 16;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // bounded waits: 2 s

constexpr int kSlotBadPos = -1, kSlotPadding = -2;

// Per token of the tile: where its rows go, and its angle's position.
struct TokenDest {
  int page;  // pool page, or -1
  int slot;  // slot of the page, or kSlotBadPos / kSlotPadding
  int pos;   // position of the angle
  int pad;
};

__host__ __device__ inline int round16(int n) { return (n + 15) & ~15; }

// Rows of one kind, padded to whole warp stages.
__host__ __device__ inline size_t tile_smem(int tokens, int heads, int group, bool with_q) {
  const int nk = round16(tokens * heads), nq = with_q ? round16(tokens * heads * group) : 0;
  return static_cast<size_t>(2 * nk + nq) * kRow + static_cast<size_t>(tokens) * (2 * (kD / 2) * 4 + sizeof(TokenDest)) + 16;
}

// Two 16-bit values of a word -> fp32 pair, exact.
template <bool BF16>
__device__ __forceinline__ f2 widen(uint32_t w) {
  if constexpr (BF16) return pk(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  else return pk(cvt_f16(w & 0xFFFFu), cvt_f16(w >> 16));
}

// Position rotation of one lane's half row.  row: the row in shared memory; raw[t] = its chunk
// t ^ rho (of the lane's half l); cs: the token's cosines [64], then sines [64]; x[4t + e] =
// channels 2e, 2e + 1 of chunk t ^ rho after the rotation.  Chunks are 8 channels and
// rotary_dim is a multiple of 16, so a chunk's partner is a whole chunk.
template <bool BF16>
__device__ __forceinline__ void rope_row(const uint4 (&raw)[8], uint32_t row, uint32_t cs, int rho, int l,
                                         const RopeAppendParams& p, f2 (&x)[32]) {
  const int half = p.rotary_dim >> 4;  // chunks in half of the rotated channels
#pragma unroll
  for (int t = 0; t < 8; t++) {
    const int c = 8 * l + (t ^ rho);
    const uint32_t w[4] = {raw[t].x, raw[t].y, raw[t].z, raw[t].w};
#pragma unroll
    for (int e = 0; e < 4; e++) x[4 * t + e] = widen<BF16>(w[e]);
    if (c >= 2 * half) continue;
    if (!p.interleaved) {
      const bool lower = c < half;
      const int fc = lower ? c : c - half;
      const uint4 other = lds_128(row + 16 * (lower ? c + half : c - half));
      const uint32_t ow[4] = {other.x, other.y, other.z, other.w};
      const float sg = lower ? -1.0f : 1.0f;
      const f2 SG = pk(sg, sg);
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const uint4 cc = lds_128(cs + 32 * fc + 8 * e), ss = lds_128(cs + 256 + 32 * fc + 8 * e);
        const f2 C0 = pk(__uint_as_float(cc.x), __uint_as_float(cc.y)), C1 = pk(__uint_as_float(cc.z), __uint_as_float(cc.w));
        const f2 S0 = pk(__uint_as_float(ss.x), __uint_as_float(ss.y)), S1 = pk(__uint_as_float(ss.z), __uint_as_float(ss.w));
        // fma(fl(other s), +-1, fl(own c)): the sum or difference with one rounding
        x[4 * t + e] = fma2(mul2(widen<BF16>(ow[e]), S0), SG, mul2(x[4 * t + e], C0));
        x[4 * t + e + 1] = fma2(mul2(widen<BF16>(ow[e + 1]), S1), SG, mul2(x[4 * t + e + 1], C1));
      }
    } else {
      const uint4 cc = lds_128(cs + 16 * c), ss = lds_128(cs + 256 + 16 * c);
      const float cf[4] = {__uint_as_float(cc.x), __uint_as_float(cc.y), __uint_as_float(cc.z), __uint_as_float(cc.w)};
      const float sf[4] = {__uint_as_float(ss.x), __uint_as_float(ss.y), __uint_as_float(ss.z), __uint_as_float(ss.w)};
#pragma unroll
      for (int e = 0; e < 4; e++) {
        float a, b;
        upk(x[4 * t + e], a, b);
        x[4 * t + e] = fma2(mul2(pk(b, a), pk(sf[e], sf[e])), pk(-1.0f, 1.0f), mul2(x[4 * t + e], pk(cf[e], cf[e])));
      }
    }
  }
}

template <int BLOCK, bool FP4, bool BF16>
__global__ void __launch_bounds__(kThreads, 4) rope_append_kernel(RopeAppendParams p) {
  griddep_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int t0 = blockIdx.x * p.tile_tokens, nt = min(p.tile_tokens, p.total_new_tokens - t0);
  const int h0 = blockIdx.y * p.tile_heads, nh = min(p.tile_heads, p.num_kv_heads - h0);
  const int gq = p.q ? nh * p.group : 0;  // q rows per token of this CTA
  const int nk = nt * nh, nq = nt * gq;
  // [K rows][V rows][q rows], each padded to 16 rows | cosines and sines | destinations | barrier
  const uint32_t base = smem_addr(smem);
  const uint32_t k_s = base, v_s = k_s + round16(nk) * kRow, q_s = v_s + round16(nk) * kRow;
  uint8_t* const tail = smem + (2 * round16(nk) + round16(nq)) * kRow;
  float* const cs = reinterpret_cast<float*>(tail);
  TokenDest* const dest = reinterpret_cast<TokenDest*>(cs + nt * kD);
  const uint32_t bar = smem_addr(dest + nt);
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  griddep_wait();
  if (tid == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(2 * nk + nq) * kRow);
  __syncthreads();
  // One bulk copy per token and kind: a token's heads are contiguous.
  for (int i = tid; i < 3 * nt; i += kThreads) {
    const int kind = i / nt, t = i - kind * nt;
    if (kind == 2 && nq == 0) continue;
    const int rows = kind == 2 ? gq : nh;
    const uint8_t* src = static_cast<const uint8_t*>(kind == 0 ? p.k : kind == 1 ? p.v : p.q);
    const int64_t stride = kind == 0 ? p.k_stride : kind == 1 ? p.v_stride : p.q_stride;
    src += (static_cast<int64_t>(t0 + t) * stride) * 2 + static_cast<int64_t>(kind == 2 ? h0 * p.group : h0) * kRow;
    const uint32_t dst = (kind == 0 ? k_s : kind == 1 ? v_s : q_s) + t * rows * kRow;
    bulk_copy_g2s(dst, src, rows * kRow, bar, l2_policy_evict_first());
  }
  // Each token's sequence, destination and position.
  for (int i = tid; i < nt; i += kThreads) {
    const int t = t0 + i;
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu_new_tokens + mid) <= t) lo = mid; else hi = mid;
    }
    const int first = __ldg(p.cu_new_tokens + lo);
    TokenDest d = {-1, kSlotPadding, 0, 0};
    if (t >= first && t < __ldg(p.cu_new_tokens + lo + 1)) {
      const long long pos = static_cast<long long>(__ldg(p.seq_lens + lo)) + (t - first);
      d.pos = p.positions ? __ldg(p.positions + t) : static_cast<int>(pos);
      d.slot = kSlotBadPos;
      if (pos >= 0 && (pos >> p.page_shift) < p.max_pages_per_seq) {
        d.slot = static_cast<int>(pos) & (p.page_size - 1);
        d.page = __ldg(p.page_table + static_cast<size_t>(lo) * p.max_pages_per_seq + (pos >> p.page_shift));
      }
      if (d.slot < 0) atomicOr(p.status, KVQ_DEV_BAD_POS_BIT);
      else if (d.page < 0 || d.page >= p.num_pages) {
        atomicOr(p.status, KVQ_DEV_BAD_PAGE_BIT);
        d.page = -1;
      }
    }
    dest[i] = d;
  }
  __syncthreads();
  const int pairs = p.rotary_dim >> 1;
  for (int i = tid; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, f = i - t * pairs;
    double s, c;
    sincos(static_cast<double>(dest[t].pos) * static_cast<double>(__ldg(p.inv_freq + f)), &s, &c);
    cs[t * kD + f] = static_cast<float>(c * p.factor);
    cs[t * kD + kD / 2 + f] = static_cast<float>(s * p.factor);
  }
  const bool landed = mbar_wait_bounded(bar, 0, kWaitLimitNs);
  if (!landed) {
    // Flag it; give the copies in flight another bounded wait before the CTA may exit.
    if (lane == 0) atomicOr(p.status, KVQ_DEV_TIMEOUT_BIT);
    mbar_wait_bounded(bar, 0, kWaitLimitNs);
  }
  if (__syncthreads_or(!landed)) return;

  const int l = lane & 1, rho = lane & 7;
  const unsigned pmask = 0x3u << (lane & 30);
  const int nsk = round16(nk) / kStageRows, nsq = round16(nq) / kStageRows;
  const uint32_t cs_s = smem_addr(cs);
  for (int st = w; st < 2 * nsk + nsq; st += kWarps) {
    const int kind = st < nsk ? 0 : st < 2 * nsk ? 1 : 2;
    const int r = (st - (kind == 0 ? 0 : kind == 1 ? nsk : 2 * nsk)) * kStageRows + (lane >> 1);
    const uint32_t row = (kind == 0 ? k_s : kind == 1 ? v_s : q_s) + r * kRow;
    const bool active = r < (kind == 2 ? nq : nk);
    uint4 raw[8];
    f2 x[32];
    int ti = 0;
    if (active) {  // both lanes of a row take the same branch
      ti = r / (kind == 2 ? gq : nh);
#pragma unroll
      for (int t = 0; t < 8; t++) raw[t] = lds_128(row + kD * l + 16 * (t ^ rho));
    }
    if (kind == 2) {
      uint32_t o[32];
      if (active) {
        rope_row<BF16>(raw, row, cs_s + ti * (kD * 4), rho, l, p, x);
#pragma unroll
        for (int i = 0; i < 32; i++) {
          float a, b;
          upk(x[i], a, b);
          o[i] = pack_half2(__float2half_rn(a), __float2half_rn(b));
        }
      }
      // Back into the row's place (both lanes have read both halves), then out in whole rows.
      __syncwarp();
      if (active) {
#pragma unroll
        for (int t = 0; t < 8; t++)
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(row + kD * l + 16 * (t ^ rho)), "r"(o[4 * t]),
                       "r"(o[4 * t + 1]), "r"(o[4 * t + 2]), "r"(o[4 * t + 3])
                       : "memory");
      }
      __syncwarp();
      const int r0 = (st - 2 * nsk) * kStageRows;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int rr = r0 + 2 * i + (lane >> 4);
        if (rr >= nq) continue;
        const int tt = rr / gq;
        if (dest[tt].slot == kSlotPadding) continue;
        const uint4 v = lds_128(q_s + rr * kRow + 16 * (lane & 15));
        __half* dst = p.q_out + (static_cast<size_t>(t0 + tt) * p.num_kv_heads * p.group + h0 * p.group + (rr - tt * gq)) * kD;
        stg_128(reinterpret_cast<uint8_t*>(dst) + 16 * (lane & 15), v.x, v.y, v.z, v.w);
      }
      continue;
    }
    if (active) {
      if (kind == 0) {
        rope_row<BF16>(raw, row, cs_s + ti * (kD * 4), rho, l, p, x);
      } else {
#pragma unroll
        for (int t = 0; t < 8; t++) {
          const uint32_t wd[4] = {raw[t].x, raw[t].y, raw[t].z, raw[t].w};
#pragma unroll
          for (int e = 0; e < 4; e++) x[4 * t + e] = widen<BF16>(wd[e]);
        }
      }
      if constexpr (BLOCK > 1) {
        // Stage h = 1: (a, c) -> (a + c, a - c).
#pragma unroll
        for (int i = 0; i < 32; i++) {
          float a, c;
          upk(x[i], a, c);
          x[i] = pk(__fadd_rn(a, c), __fsub_rn(a, c));
        }
      }
      rotate_stages<BLOCK>(rho, l, pmask, x);
      uint32_t q[8], sbits;
      if constexpr (FP4) sbits = quantise_fp4(x, p.cb, rho, q);
      else sbits = quantise(x, p.cb, pmask, q);
      // Codes into channel order through the row's own place in shared memory.
      __syncwarp(pmask);
      const uint32_t stg = row + 32 * l;
#pragma unroll
      for (int t = 0; t < 8; t++) sts_32(stg + 4 * (t ^ rho), q[t]);
      const uint4 c0 = lds_128(stg), c1 = lds_128(stg + 16);
      const TokenDest d = dest[ti];
      if (d.slot >= 0 && d.page >= 0) {
        const int S = p.page_size, h = h0 + (r - ti * nh);
        constexpr int kScaleBytes = FP4 ? kD / 16 : 2;
        uint8_t* blk = p.pool_layer + (static_cast<size_t>(d.page) * p.num_kv_heads + h) *
                                          (static_cast<size_t>(S) * (kD + 2 * kScaleBytes));
        uint4* crow = reinterpret_cast<uint4*>(blk + (static_cast<size_t>(kind) * S + d.slot) * (kD / 2) + 32 * l);
        crow[0] = c0;
        crow[1] = c1;
        uint8_t* srow = blk + static_cast<size_t>(S) * kD + (static_cast<size_t>(kind) * S + d.slot) * kScaleBytes;
        if constexpr (FP4) *reinterpret_cast<uint32_t*>(srow + 4 * l) = sbits;
        else if (l == 0) *reinterpret_cast<uint16_t*>(srow) = static_cast<uint16_t>(sbits);
      }
    }
  }
}

template <int BLOCK, bool FP4, bool BF16>
int launch_one(const cudaLaunchConfig_t& cfg, const RopeAppendParams& p) {
  if (!ensure_smem<rope_append_kernel<BLOCK, FP4, BF16>>(kMaxSmem)) return -2;
  return cudaLaunchKernelEx(&cfg, rope_append_kernel<BLOCK, FP4, BF16>, p) == cudaSuccess ? 0 : -2;
}

template <bool FP4, bool BF16>
int launch_block(const cudaLaunchConfig_t& cfg, const RopeAppendParams& p, int block) {
  switch (block) {
    case 1: return launch_one<1, FP4, BF16>(cfg, p);
    case 32: return launch_one<32, FP4, BF16>(cfg, p);
    case 64: return launch_one<64, FP4, BF16>(cfg, p);
    case 128: return launch_one<128, FP4, BF16>(cfg, p);
    default: return -1;
  }
}

}  // namespace

int launch_rope_append(RopeAppendParams p, int block, bool fp4, bool bf16, int num_sms, cudaStream_t stream) {
  if (p.total_new_tokens == 0) return 0;
  const int per_head = 2 + (p.q ? p.group : 0);
  int heads = kTileRows / per_head;
  if (heads > p.num_kv_heads) heads = p.num_kv_heads;
  int tokens = kTileRows / (per_head * heads);
  if (tokens > kRopeTokens) tokens = kRopeTokens;
  // A short call is spread over the SMs: tiles of fewer tokens, then of fewer heads.
  auto ctas = [&] {
    return static_cast<long long>((p.total_new_tokens + tokens - 1) / tokens) * ((p.num_kv_heads + heads - 1) / heads);
  };
  while (tokens > 1 && ctas() < 2 * num_sms) tokens = (tokens + 1) / 2;
  while (heads > 1 && ctas() < num_sms) heads = (heads + 1) / 2;
  p.tile_tokens = tokens;
  p.tile_heads = heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.total_new_tokens + tokens - 1) / tokens, (p.num_kv_heads + heads - 1) / heads);
  if (cfg.gridDim.y > 65535) return -1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = tile_smem(tokens, heads, p.group, p.q != nullptr);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (fp4) return bf16 ? launch_block<true, true>(cfg, p, block) : launch_block<true, false>(cfg, p, block);
  return bf16 ? launch_block<false, true>(cfg, p, block) : launch_block<false, false>(cfg, p, block);
}

}  // namespace kvq
