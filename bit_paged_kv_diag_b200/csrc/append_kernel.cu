// append_kernel.cu -- fused block-diagonal Hadamard rotation + token-wise INT4
// quantisation + paged append, for sm_100a.
//
// Method: "KVキャッシュを4ビットへ — SAW-INT4とシステムを踏まえたINT4量子化"
// (youngju.dev), sections "回転のトリック — ブロック対角アダマール" (rotation inside
// blocks of channels), "素朴なINT4はなぜ崩れるのか" (one scale per token, quantised
// as the token is produced) and "システムこそが設計である — 融合カーネル" (one fused
// kernel that rotates, quantises and appends into paged KV blocks without revisiting
// past tokens).
//
// Work decomposition.  Every warp runs its own pipeline: a warp stage is 8 consecutive
// (token, KV head) pairs, their K rows (2 KB, contiguous in the token-packed input) and V
// rows (2 KB), brought into a ring of 3 shared-memory slots by two 1-D bulk copies (TMA
// engine, no multicast) that complete on the slot's mbarrier.  Warps take warp stages
// gw, gw + W, ... (gw = the global warp index, W = all warps of the persistent grid) and
// never wait for one another, so their serial parts (the row's scale, the stores) spread
// out in time; no register holds prefetched data.  Two lanes handle one row (the K or V
// row of one pair, 128 fp16 channels): lane l holds channels [64l, 64l + 64) as 8 chunks
// of 8 channels.
//
// Bank-conflict-free reads.  A lane reads its chunks in the order c = t ^ rho (t = 0..7,
// rho = lane & 7): the 8 lanes of a quarter warp then touch 8 different 16-byte bank
// groups.  Register slot t holds chunk t ^ rho, so the butterfly stages that pair chunks
// (h = 8, 16, 32: chunk bits 0-2) pair slots t and t ^ k as well; whether slot t holds the
// lower or the upper chunk of the pair depends on rho, and each output is one fma with a
// +-1 multiplier (fma(a, 1, c) = a + c and fma(c, -1, a) = a - c, rounded once: the IEEE
// sum and difference).  Stages h = 1, 2, 4 are inside a chunk.  Only b = 128 has a stage
// across the lane pair (h = 64): lane 1's slot t ^ 1 holds the partner of lane 0's slot t
// (their rho differ in bit 0); after one exchange lane 0 keeps the sums (channels
// [0, 64)) and lane 1 the differences (channels [64, 128)), in the same slot order.
//
// Stages run in the fixed order h = 1, 2, ..., b/2, each pair (i, i + h) with bit h of i
// clear becoming (a + c, a - c) as one IEEE fp32 add and one subtract, then one multiply
// by the fp32 constant nearest 1/sqrt(b): rotated values are bit-exact with any
// implementation of that fixed-order butterfly.  Pairs of channels go through the packed
// fp32x2 arithmetic of sm_100 (each half is still one IEEE operation) held in 64-bit
// registers; fp16 -> fp32 conversion rides in the first stage's mixed-precision adds.
//
// Quantisation: m = max |y| (lane-pair shuffle), s = fp16_rn(m / 7) (IEEE division, once
// per row).  Codes are round-half-even of y / s, clamped to [-8, 7], computed without
// dividing: a fast multiply-by-reciprocal path, and an exact half-point comparison for
// groups with a near-tie (see quantise()); codes stay bit-exact with division by the
// stored fp16 scale.  Codes are packed two per byte (low nibble = even channel).  A
// lane's 8 code words (one per chunk, in slot order) go through a per-warp staging area
// in shared memory, written at their chunk's place and read back in channel order, so
// that the row's 64 code bytes leave as two 16-byte stores per lane (one L2 request per
// row and store); lane 0 of the row stores the scale.
//
// NVFP4 rows ("BitDecoding-FP4:FP4 KVキャッシュのネイティブ復号" (sns.style), sections
// "背景と概要", "深掘り分析": 4-bit microscaling elements with E4M3 block scales): after
// the same rotation, each block of 16 channels -- slots t and t ^ 1 of a lane, since the
// rotation of the read order keeps chunk pairs together -- gets s = E4M3(fl(max|y| / 6))
// (round to nearest even, saturated at 448) and codes E2M1(fl(y * fl(1/s))) (nearest
// even, saturated at 6, sign kept), both by the hardware conversions cvt.rn.satfinite;
// all codes 0 when s == 0.  A lane's 4 scale bytes are stored as one word.
#include <cuda_fp16.h>
#include <stdint.h>

#include "append_row.cuh"
#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

namespace {

constexpr int kD = 128;
constexpr int kPairs = 8;                      // (token, KV head) pairs per warp stage
constexpr int kWarps = 8;                      // warps per CTA
constexpr int kThreads = 32 * kWarps;
constexpr int kHalfBytes = kPairs * kD * 2;    // one tensor's rows of a warp stage: 2 KB
constexpr int kSlotBytes = 2 * kHalfBytes;     // K rows, then V rows
constexpr int kStages = 3;                     // ring slots per warp
constexpr int kStgStride = 80;                 // staging bytes per row (64 used)
// A warp's region: ring slots | staging lines | sequence cursors (16 B per pair slot) |
// barriers, rounded to 128 bytes so that every region (and so every copy destination)
// stays 16-byte aligned.
constexpr int kCursorBytes = 16 * kPairs;
constexpr int kWarpBytes =
    (kStages * kSlotBytes + 2 * kPairs * kStgStride + kCursorBytes + 8 * kStages + 127) / 128 * 128;
constexpr int kSmemBytes = kWarps * kWarpBytes;
constexpr int kCtasPerSm = 2;
static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM must fit");
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // bounded waits: 2 s

// Issue the two bulk copies of warp stage j (pairs [8j, 8j + n)) into the slot at dst.
__device__ __forceinline__ void issue_stage(const AppendParams& p, int j, int npairs,
                                            uint32_t dst, uint32_t bar, uint64_t pol) {
  const int g0 = j * kPairs;
  const int left = npairs - g0;
  const uint32_t bytes = static_cast<uint32_t>(left < kPairs ? left : kPairs) * (kD * 2);
  mbar_arrive_expect_tx(bar, 2 * bytes);
  bulk_copy_g2s(dst, p.k + static_cast<size_t>(g0) * kD, bytes, bar, pol);
  bulk_copy_g2s(dst + kHalfBytes, p.v + static_cast<size_t>(g0) * kD, bytes, bar, pol);
}

// Where pair gp goes: its sequence b (the b with cu[b] <= t < cu[b+1]), position pos =
// seq_lens[b] + t - cu[b], the raw page-table entry of page pos / S (checked at use, so
// that the load is in flight meanwhile) and the slot pos % S, or slot -1 for a position
// outside the page table.
struct Dest {
  int page;
  int slot;
  int h;
};

// The sequence of a pair slot's current token, kept in shared memory across the warp's
// stages (whose tokens only increase) as {b, cu_lo, cu_hi, sl}: [cu_lo, cu_hi) = the
// sequence's tokens in the call, sl = its length before the call.  A token outside the
// range moves the cursor by a binary search over cu_new_tokens; a token inside it needs no
// global load.  The four lanes of a pair read and write the same entry with the same
// values; the warp syncs between stages.
__device__ __forceinline__ Dest pair_dest(const AppendParams& p, int gp, uint32_t cursor) {
  Dest d;
  // t = gp / num_kv_heads by the host's multiplier (gp < 2^31); pos / S and pos % S by
  // the power-of-two page size.
  const int t = static_cast<int>(__umulhi(static_cast<uint32_t>(gp) << 1, p.heads_magic) >> p.heads_shift);
  d.h = gp - t * p.num_kv_heads;
  uint4 sc = lds_128(cursor);  // x = b, y = cu_lo, z = cu_hi, w = sl
  if (t < static_cast<int>(sc.y) || t >= static_cast<int>(sc.z)) {
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu_new_tokens + mid) <= t) lo = mid; else hi = mid;
    }
    sc = make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(__ldg(p.cu_new_tokens + lo)),
                    static_cast<uint32_t>(__ldg(p.cu_new_tokens + lo + 1)),
                    static_cast<uint32_t>(__ldg(p.seq_lens + lo)));
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(cursor), "r"(sc.x), "r"(sc.y), "r"(sc.z),
                 "r"(sc.w)
                 : "memory");
  }
  const int b = static_cast<int>(sc.x);
  const int pos = static_cast<int>(sc.w) + (t - static_cast<int>(sc.y));
  const int lp = pos >= 0 ? pos >> p.page_shift : 0;
  if (pos < 0 || lp >= p.max_pages_per_seq) {
    d.page = -1;
    d.slot = -1;
  } else {
    d.page = __ldg(p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq + lp);
    d.slot = pos & (p.page_size - 1);
  }
  return d;
}

// A finished row to its place in the pool: the lane's 32 code bytes (c0, c1) and the row's scale;
// a bad position or page is flagged and not stored.
template <bool FP4>
__device__ __forceinline__ void store_row(const AppendParams& p, const Dest& dcur, int kv, int l, uint4 c0, uint4 c1,
                                          uint32_t sbits) {
  const bool bad_pos = dcur.slot < 0;
  if (bad_pos || dcur.page < 0 || dcur.page >= p.num_pages) {
    if (l == 0 && kv == 0)
      atomicOr(p.status, bad_pos ? KVQ_DEV_BAD_POS_BIT : KVQ_DEV_BAD_PAGE_BIT);
  } else {
    const int S = p.page_size;
    constexpr int kScaleBytes = FP4 ? kD / 16 : 2;  // per token row
    uint8_t* blk = p.pool_layer + (static_cast<size_t>(dcur.page) * p.num_kv_heads + dcur.h) *
                                      (static_cast<size_t>(S) * (kD + 2 * kScaleBytes));
    uint4* crow = reinterpret_cast<uint4*>(blk + static_cast<size_t>(kv) * S * (kD / 2) +
                                           static_cast<size_t>(dcur.slot) * (kD / 2) + 32 * l);
    crow[0] = c0;
    crow[1] = c1;
    uint8_t* srow = blk + static_cast<size_t>(S) * kD + static_cast<size_t>(kv) * S * kScaleBytes +
                    static_cast<size_t>(dcur.slot) * kScaleBytes;
    if constexpr (FP4) {
      *reinterpret_cast<uint32_t*>(srow + 4 * l) = sbits;
    } else {
      if (l == 0) *reinterpret_cast<uint16_t*>(srow) = static_cast<uint16_t>(sbits);
    }
  }
}

template <int BLOCK, bool FP4>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) append_kernel(AppendParams p) {
  // The next kernel may start its own prologue; the row copies and the pool stores below wait
  // for every earlier kernel (griddep_wait): it may be writing these rows or reading the pool.
  griddep_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  // This warp's ring, staging lines and barriers.
  const uint32_t ring = smem_addr(smem) + w * kWarpBytes;
  const uint32_t stg = ring + kStages * kSlotBytes;
  const uint32_t cursors = stg + 2 * kPairs * kStgStride;
  const uint32_t bar0 = cursors + kCursorBytes;
  const int l = lane & 1, rho = lane & 7;
  const int pr = lane >> 2;         // pair within the warp stage
  const int kv = (lane >> 1) & 1;   // 0 = K row, 1 = V row
  // Shuffles never leave the lane pair of a row, so they name only those two lanes.
  const unsigned pmask = 0x3u << (lane & 30);
  const int npairs = p.total_new_tokens * p.num_kv_heads;  // < 2^31 (host-checked)
  const int nws = (npairs + kPairs - 1) / kPairs;
  const int W = gridDim.x * kWarps;
  const int gw = blockIdx.x * kWarps + w;
  // This row's 80-byte staging line; the lane's half is at +32l.
  const uint32_t stg_row = stg + (lane >> 1) * kStgStride + 32 * l;
  const uint64_t pol = l2_policy_evict_first();

  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; s++) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
    griddep_wait();  // (the other lanes: before their first store)
#pragma unroll
    for (int s = 0; s < kStages; s++) {
      const int j = gw + s * W;
      if (j < nws) issue_stage(p, j, npairs, ring + s * kSlotBytes, bar0 + 8 * s, pol);
    }
  }
  __syncwarp();

  const uint32_t cursor = cursors + 16 * pr;  // this lane's pair slot
  if ((lane & 3) == 0)  // an empty range: the first lookup searches
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(cursor), "r"(0u) : "memory");
  __syncwarp();
  Dest dcur = {-1, -1, 0};
  if (gw * kPairs + pr < npairs) dcur = pair_dest(p, gw * kPairs + pr, cursor);
  bool waited = false;
  int s = 0;
  uint32_t phase = 0;
  for (int j = gw; j < nws; j += W) {
    const uint32_t slot = ring + s * kSlotBytes;
    const int gp = j * kPairs + pr;
    const bool active = gp < npairs;
    // The next warp stage's destination: its page-table load is in flight meanwhile.
    Dest dnext = {-1, -1, 0};
    if (j + W < nws && gp + W * kPairs < npairs) dnext = pair_dest(p, gp + W * kPairs, cursor);

    if (!mbar_wait_warp(bar0 + 8 * s, phase, kWaitLimitNs)) {
      // A copy did not land in time: flag it, give it and this warp's other copies another
      // (bounded) wait so that nothing lands in shared memory after the CTA exits, and stop.
      if (lane == 0) atomicOr(p.status, KVQ_DEV_TIMEOUT_BIT);
#pragma unroll
      for (int k = 0; k < kStages; k++) {
        const int sk = (s + k) % kStages;
        if (j + k * W < nws)
          mbar_wait_warp(bar0 + 8 * sk, sk >= s ? phase : phase ^ 1u, kWaitLimitNs);
      }
      return;
    }
    uint4 raw[8];
    if (active) {
      const uint32_t row = slot + kv * kHalfBytes + pr * (kD * 2) + l * kD;
#pragma unroll
      for (int t = 0; t < 8; t++) raw[t] = lds_128(row + 16 * (t ^ rho));
    }
    // Every read of this slot is done: it can take warp stage j + kStages * W.
    __syncwarp();
    if (lane == 0 && j + kStages * W < nws) {
      fence_proxy_async_smem();
      issue_stage(p, j + kStages * W, npairs, slot, bar0 + 8 * s, pol);
    }
    if (++s == kStages) {
      s = 0;
      phase ^= 1u;
    }

    if (active) {  // both lanes of a row, and both rows of a pair, take the same branch
      f2 x[32];
      rotate_row<BLOCK>(raw, rho, l, pmask, x);
      uint32_t q[8];
      uint32_t sbits;
      if constexpr (FP4) sbits = quantise_fp4(x, p.cb, rho, q);
      else sbits = quantise(x, p.cb, pmask, q);
      // Slot t's word is word t ^ rho of the lane's half: through the staging line into
      // channel order (the lane reads back only what it wrote).
#pragma unroll
      for (int t = 0; t < 8; t++) sts_32(stg_row + 4 * (t ^ rho), q[t]);
      const uint4 c0 = lds_128(stg_row), c1 = lds_128(stg_row + 16);
      if (!waited) {
        griddep_wait();
        waited = true;
      }
      store_row<FP4>(p, dcur, kv, l, c0, c1, sbits);
    }
    dcur = dnext;
  }
}

// The same for a call of at most one warp stage per warp and one CTA per SM (decode steps, short
// chunks), where a launch is a chain of latencies: the rows are copied and quantised before the wait
// for the previous kernel, under its tail.  That kernel may be the one that writes these rows (a
// read-back, say), so a warp of its own waits and copies them again, next to the arithmetic where
// there is nothing to wait for; a stage is stored if both copies are the same, and otherwise done again
// on the second.  An append and a decode in turn (16 x 4096 tokens, in a graph): 25.7 us; with the copies
// after the wait 28.4; with no second copy, right only if no kernel of this library writes the rows, 24.5.
template <int BLOCK, bool FP4>
__global__ void __launch_bounds__(kThreads + 32, 1) append_few_kernel(AppendParams p) {
  griddep_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int npairs = p.total_new_tokens * p.num_kv_heads;
  const int nws = (npairs + kPairs - 1) / kPairs;
  const uint64_t pol = l2_policy_evict_first();
  // Warp ww's region, as in append_kernel: slots 0 and 1 take the first and the second copy.
  auto region = [&](int ww) { return smem_addr(smem) + ww * kWarpBytes; };
  constexpr int kCursors = kStages * kSlotBytes + 2 * kPairs * kStgStride, kBars = kCursors + kCursorBytes;
  const int j = blockIdx.x * kWarps + w;
  const bool have = w < kWarps && j < nws;
  if (have && lane == 0) {
    mbar_init(region(w) + kBars, 1);
    mbar_init(region(w) + kBars + 8, 1);
    fence_mbar_init();
    issue_stage(p, j, npairs, region(w), region(w) + kBars, pol);
  }
  __syncthreads();
  if (w == kWarps) {
    griddep_wait();
    const int jj = blockIdx.x * kWarps + lane;
    if (lane < kWarps && jj < nws)
      issue_stage(p, jj, npairs, region(lane) + kSlotBytes, region(lane) + kBars + 8, pol);
    return;
  }
  if (!have) return;

  const int l = lane & 1, rho = lane & 7, pr = lane >> 2, kv = (lane >> 1) & 1;
  const unsigned pmask = 0x3u << (lane & 30);
  const uint32_t ring = region(w), bar0 = ring + kBars, cursor = ring + kCursors + 16 * pr;
  const uint32_t stg_row = ring + kStages * kSlotBytes + (lane >> 1) * kStgStride + 32 * l;
  const uint32_t row = ring + kv * kHalfBytes + pr * (kD * 2) + l * kD;  // of the first copy
  if ((lane & 3) == 0)  // an empty range: the lookup searches
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(cursor), "r"(0u) : "memory");
  __syncwarp();
  const bool active = j * kPairs + pr < npairs;
  Dest d = {-1, -1, 0};
  if (active) d = pair_dest(p, j * kPairs + pr, cursor);
  bool late = !mbar_wait_warp(bar0, 0u, kWaitLimitNs);
  uint4 c0 = make_uint4(0u, 0u, 0u, 0u), c1 = c0;
  uint32_t sbits = 0u;
#pragma unroll 1
  for (int copy = 0; !late; copy++) {
    if (active) {  // both lanes of a row, and both rows of a pair, take the same branch
      uint4 raw[8];
#pragma unroll
      for (int t = 0; t < 8; t++) raw[t] = lds_128(row + copy * kSlotBytes + 16 * (t ^ rho));
      f2 x[32];
      rotate_row<BLOCK>(raw, rho, l, pmask, x);
      uint32_t q[8];
      if constexpr (FP4) sbits = quantise_fp4(x, p.cb, rho, q);
      else sbits = quantise(x, p.cb, pmask, q);
#pragma unroll
      for (int t = 0; t < 8; t++) sts_32(stg_row + 4 * (t ^ rho), q[t]);
      c0 = lds_128(stg_row);
      c1 = lds_128(stg_row + 16);
    }
    if (copy) break;
    griddep_wait();
    late = !mbar_wait_warp(bar0 + 8, 0u, kWaitLimitNs);
    uint32_t diff = 0u;
    if (active) {
#pragma unroll
      for (int t = 0; t < 8; t++) {
        const uint4 a = lds_128(row + 16 * (t ^ rho)), b = lds_128(row + kSlotBytes + 16 * (t ^ rho));
        diff |= (a.x ^ b.x) | (a.y ^ b.y) | (a.z ^ b.z) | (a.w ^ b.w);
      }
    }
    if (!__any_sync(0xffffffffu, diff != 0u)) break;
  }
  if (late) {
    // A copy did not land in time: as in append_kernel.
    if (lane == 0) atomicOr(p.status, KVQ_DEV_TIMEOUT_BIT);
    mbar_wait_warp(bar0, 0u, kWaitLimitNs);
    mbar_wait_warp(bar0 + 8, 0u, kWaitLimitNs);
    return;
  }
  if (active) store_row<FP4>(p, d, kv, l, c0, c1, sbits);
}

template <int BLOCK, bool FP4>
int launch_block(const cudaLaunchConfig_t& cfg, const AppendParams& p, bool few) {
  if (few) {
    if (!ensure_smem<append_few_kernel<BLOCK, FP4>>(kSmemBytes)) return -2;
    return cudaLaunchKernelEx(&cfg, append_few_kernel<BLOCK, FP4>, p) == cudaSuccess ? 0 : -2;
  }
  if (!ensure_smem<append_kernel<BLOCK, FP4>>(kSmemBytes)) return -2;
  return cudaLaunchKernelEx(&cfg, append_kernel<BLOCK, FP4>, p) == cudaSuccess ? 0 : -2;
}

template <bool FP4>
int launch_format(const cudaLaunchConfig_t& cfg, const AppendParams& p, int block, bool few) {
  switch (block) {
    case 1: return launch_block<1, FP4>(cfg, p, few);
    case 32: return launch_block<32, FP4>(cfg, p, few);
    case 64: return launch_block<64, FP4>(cfg, p, few);
    case 128: return launch_block<128, FP4>(cfg, p, few);
    default: return -1;
  }
}

}  // namespace

int launch_append(const AppendParams& p, int block, int num_sms, cudaStream_t stream) {
  const long long npairs = static_cast<long long>(p.total_new_tokens) * p.num_kv_heads;
  if (npairs == 0) return 0;
  if (npairs > 0x7fffffffLL - (64LL << 20)) return -1;  // int indexing in the kernel
  const long long nws = (npairs + kPairs - 1) / kPairs;
  // One wave of persistent CTAs, or fewer for a small call.
  const long long full = static_cast<long long>(kCtasPerSm) * num_sms;
  const long long need = (nws + kWarps - 1) / kWarps;
  const long long grid = need < full ? need : full;
  const bool few = need <= num_sms;  // at most a warp stage per warp and a CTA per SM
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(few ? kThreads + 32 : kThreads);  // (and the warp that copies again)
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.fp4 ? launch_format<true>(cfg, p, block, few) : launch_format<false>(cfg, p, block, few);
}

}  // namespace kvq
