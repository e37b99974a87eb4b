// sparse_attention.cu -- attention over chosen pages of the paged 4-bit cache, for sm_100a: each
// query and KV head reads the pages of its own list, and nothing else of the cache.
//
// Mathematics.  For query t at position p of its sequence and KV head h, softmax attention of
// the G query heads over the tokens at or before p of the pages blocks[t][h][0 .. num_blocks)
// (negative entries are empty; a list that leaves no token gives zeros), with the decode
// kernel's arithmetic (decode_tile.cuh): q rotated and carried in full precision, scores exact
// in integers (INT4) or f16 MMAs (NVFP4), the softmax in one pass with running maximum and sum,
// the output rotated back and rounded once.
//
// Work split.  A unit is (query, KV head) and has ceil(num_blocks * S / 32) tiles of 32 tokens.
// A CTA of 4 warps takes one of `splits` equal parts of a unit; its warps take the part's tiles
// in turn through their own rings of shared-memory slots (bulk copies, one per page and piece)
// and merge in shared memory.  Tiles without a token to attend are skipped before their copy.
// With splits > 1 (few units: the parts fill the SMs), each CTA leaves one record per query head
// in the handle's scratch and the last to arrive merges them in the order of the parts, so the
// result does not depend on the order of arrival.
//
// Measured, the kernel alone behind a flush of L2: 16 sequences x 8 KV heads, G = 4, INT4, 4096 tokens
// each: 25.0 us, 2.8 TB/s (a plain stream of these 69 MB takes 14 us; the dense decode of the same
// bytes, back to back in a graph, 22.4 us); 951 queries x 4 KV heads, G = 8, NVFP4, 1024 tokens each: 201
// us, 2.8 TB/s out of L2.  Bound by instructions: about 530 a tile (INT4, G = 4) and 870 (NVFP4, G = 8),
// most of them dequantisation, at 51 and 61 % of the issue slots.  Four CTAs per SM were 4 % faster than
// three with a deeper ring although their 128 registers spill at G = 8 (stored / loaded bytes: NVFP4 156 /
// 120 with tiles of one page, 12 / 12 with two; INT4 44 / 32 and 80 / 116) and a little with tiles of two
// pages at G = 1 (INT4, 12 / 36) and G = 2 (NVFP4, 4 / 4); G = 4 does not.
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include "decode_tile.cuh"
#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

namespace {

constexpr int kMaxSplits = 8;
constexpr int kCtasPerSm = 4;
// Ring slots of a warp: four CTAs of either format fit into an SM's shared memory.
template <bool FP4>
constexpr int kRing = FP4 ? 2 : 3;

// A page of a tile, one per lane: its block's address (16-byte aligned; bits 0-2 = the tile's
// first token in the page / 32), and the tokens to attend in the tile's part of it (<= 0: none).
struct Entry {
  uint64_t addr;
  int ntok;
};

template <int SEFF>
struct Tiles {
  static constexpr int kPPT = SEFF < kTileTokens ? kTileTokens / SEFF : 1;  // pages of a tile
  static constexpr int kBatch = 32 / kPPT;                                  // tiles of a batch
};

// Where a unit's pages and limits are.
struct UnitInfo {
  const int32_t* table;  // the sequence's page-table row
  int pos;               // the query's position (-1: nothing to attend)
  int h;
};

// This lane's page (lane % kPPT) of tile x of the unit: the logical page that the list names there;
// negative: none.
template <int SEFF>
__device__ __forceinline__ int load_block(int x, int x1, int lane, const int32_t* list, const DecodeParams& p,
                                          const SparseParams& sp) {
  constexpr int kPPT = Tiles<SEFF>::kPPT;
  const int j = SEFF < kTileTokens ? x * kPPT + lane % kPPT : (x * kTileTokens) >> p.page_shift;
  return x < x1 && j < sp.num_blocks ? __ldcg(list + j) : -1;
}

// Entry of this lane: logical page blk for tile x.
template <int SEFF, bool FP4>
__device__ __forceinline__ Entry make_entry(int x, int blk, const UnitInfo& u, const DecodeParams& p) {
  Entry e = {0, 0};
  const int off = SEFF < kTileTokens ? 0 : (x * kTileTokens) & (p.page_size - 1);
  if (blk < 0 || blk > (u.pos >> p.page_shift)) return e;  // (an arithmetic shift: -1 stays below 0)
  const int left = u.pos + 1 - (blk << p.page_shift) - off;
  if (left <= 0) return e;
  const int page = __ldg(u.table + blk);
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.status, KVQ_DEV_BAD_PAGE_BIT);
    return e;
  }
  e.ntok = min(left, SEFF);
  e.addr = reinterpret_cast<uint64_t>(p.pool_layer + (static_cast<size_t>(page) * p.num_kv_heads + u.h) *
                                                         (static_cast<size_t>(p.page_size) * row_bytes(FP4))) |
           static_cast<uint64_t>(off / kTileTokens);
  return e;
}

// What one lane copies of a tile.  Pages of up to 32 tokens: lane j < kPPT the whole block of page j;
// larger pages: lanes 0-3 the tile's K codes, V codes, K scales and V scales.
struct Piece {
  uint32_t src, per_token;  // byte of the page block, and bytes for each token before the tile's first
  uint32_t dst, bytes;      // place in the slot; 0 bytes: nothing to copy
};
template <int SEFF, bool FP4>
__device__ __forceinline__ Piece piece_of(int lane, int S) {
  constexpr int kPPT = Tiles<SEFF>::kPPT;
  constexpr uint32_t SC = FP4 ? kD / 16 : 2;  // scale bytes of a row
  const uint32_t s = static_cast<uint32_t>(S);
  if (SEFF < kTileTokens || S == kTileTokens) {
    const uint32_t blk = s * row_bytes(FP4);
    return {0u, 0u, lane * blk, lane < kPPT ? blk : 0u};
  }
  if (lane == 0) return {0u, 64u, 0u, 64u * kTileTokens};
  if (lane == 1) return {s * 64, 64u, 64u * kTileTokens, 64u * kTileTokens};
  if (lane == 2) return {s * 128, SC, 128u * kTileTokens, SC * kTileTokens};
  if (lane == 3) return {s * (128 + SC), SC, (128 + SC) * kTileTokens, SC * kTileTokens};
  return {0u, 0u, 0u, 0u};
}

// Bulk copies of one tile into a ring slot (the whole warp; with one page per tile every lane holds
// its entry, with two lane j < 2 page j's).
template <int SEFF, bool FP4>
__device__ __forceinline__ void issue_tile(Entry e, const Piece& c, uint32_t slot, uint32_t bar, int lane) {
  constexpr int kPPT = Tiles<SEFF>::kPPT;
  uint32_t total = slot_bytes(FP4);
  if (kPPT == 2) total = __popc(__ballot_sync(kFull, lane < kPPT && e.ntok > 0)) * c.bytes;  // (lane 0's: one block)
  if (lane == 0) mbar_arrive_expect_tx(bar, total);
  __syncwarp();
  if (c.bytes && e.ntok > 0) {
    const uint8_t* blk = reinterpret_cast<const uint8_t*>(e.addr & ~static_cast<uint64_t>(15));
    const uint32_t off = c.src + static_cast<uint32_t>(e.addr & 7u) * kTileTokens * c.per_token;
    bulk_copy_g2s(slot + c.dst, blk + off, c.bytes, bar, 0ull);
  }
}

template <int G, int SEFF, bool FP4>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) sparse_kernel(DecodeParams p, SparseParams sp, int splits) {
  constexpr int kSlot = slot_bytes(FP4);
  constexpr int kPPT = Tiles<SEFF>::kPPT, kBatch = Tiles<SEFF>::kBatch;
  griddep_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
  uint8_t* ring = smem;                                                        // [w][stage][kSlot]
  uint8_t* qraw = ring + kWarps * kRing<FP4> * kSlot;                             // [G][128] fp16
  uint32_t* frag = reinterpret_cast<uint32_t*>(qraw + G * kD * 2);             // [frag_words]
  float* sf = reinterpret_cast<float*>(frag + frag_words(G, FP4));             // [8]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sf + 8);                        // [w][kRing<FP4>]
  __shared__ int2 valid_ring[kWarps][kRing<FP4>];  // tokens to attend of the tile in each slot
  __shared__ int last_flag;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int unit = blockIdx.x / splits, part = blockIdx.x - unit * splits;
  const int t = unit / p.num_kv_heads, h = unit - t * p.num_kv_heads;
  const uint32_t bar_s = smem_addr(bars + w * kRing<FP4>);
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kRing<FP4>; s++) mbar_init(bar_s + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();
  griddep_wait();

  // q and the first batch of the list are on their way before anything else is looked up: behind
  // the first tiles' copies they would wait for those.
  uint4 qv = make_uint4(0u, 0u, 0u, 0u);
  if (tid < G * kD / 8)
    qv = __ldcg(reinterpret_cast<const uint4*>(p.q + (static_cast<size_t>(t) * p.num_kv_heads + h) * G * kD) + tid);
  // This warp's tiles: x0 + w, x0 + w + kWarps, ... < x1.
  const int ntile = (sp.num_blocks * p.page_size + kTileTokens - 1) / kTileTokens;
  const int x0 = static_cast<int>(static_cast<long long>(ntile) * part / splits);
  const int x1 = static_cast<int>(static_cast<long long>(ntile) * (part + 1) / splits);
  const int nT = max(0, (x1 - x0 - w + kWarps - 1) / kWarps);
  const int32_t* const list = sp.blocks + static_cast<size_t>(unit) * sp.num_blocks;
  const int xl = x0 + w + kWarps * (lane / kPPT);  // this lane's tile of the first batch
  const int blk0 = load_block<SEFF>(xl, x1, lane, list, p, sp);

  // The query's sequence and position.  A sequence is good or bad as a whole: every row of one that
  // is shorter than its chunk or does not fit its table is zeros.
  int b = t, len, pos, fewest = 0;
  if (sp.cu_q) {
    int first, end;
    const SeqWindow win = seq_window(sp.cu_q, p.batch, t);
    b = seq_find(win, sp.cu_q, p.batch, t, first, end);
    if (t < first || t >= end) return;  // a row of no sequence: left as it is
    len = __ldg(p.seq_lens + b);
    pos = len - (end - t);
    fewest = end - first;
  } else {
    len = __ldg(p.seq_lens + b);
    pos = len - 1;
  }
  if (len < fewest || len > static_cast<long long>(p.max_pages_per_seq) * p.page_size) {
    if (tid == 0) atomicOr(p.status, KVQ_DEV_BAD_POS_BIT);
    pos = -1;
  }
  UnitInfo u;
  u.table = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;
  u.pos = pos;
  u.h = h;

  uint8_t* const ring_w = ring + w * kRing<FP4> * kSlot;
  const uint32_t ring_s = smem_addr(ring_w);
  // Producer: batches of kBatch tiles; `todo` holds the batch's tiles that have a token.
  int tb = -kBatch;
  unsigned todo = 0;
  Entry cur = {0, 0};
  auto fetch = [&](int first) {
    const int x = xl + kWarps * first;
    return make_entry<SEFF, FP4>(x, load_block<SEFF>(x, x1, lane, list, p, sp), u, p);
  };
  Entry nxt = make_entry<SEFF, FP4>(xl, blk0, u, p);
  int issued = 0, next_slot = 0;
  const Piece piece = piece_of<SEFF, FP4>(lane, p.page_size);
  auto produce = [&]() {  // issue the next tile that has a token, if any
    while (todo == 0) {
      tb += kBatch;
      if (tb >= nT) return;
      cur = nxt;
      nxt = tb + kBatch < nT ? fetch(tb + kBatch) : Entry{0, 0};
      todo = __ballot_sync(kFull, cur.ntok > 0);
      if (kPPT == 2) todo = (todo | (todo >> 1)) & 0x55555555u;
    }
    const int i = __ffs(todo) - 1;  // lane of the tile's first page
    todo &= todo - 1;
    const int from = kPPT == 2 ? (i + (lane & 1)) & 31 : i;
    Entry e;
    e.addr = __shfl_sync(kFull, cur.addr, from);
    e.ntok = __shfl_sync(kFull, cur.ntok, from);
    const int s = next_slot;
    next_slot = s + 1 == kRing<FP4> ? 0 : s + 1;
    if (kPPT == 2) {
      if (lane < 2) reinterpret_cast<int*>(&valid_ring[w][s])[lane] = e.ntok;
    } else if (lane == 0) {
      valid_ring[w][s] = make_int2(e.ntok, e.ntok - 16);
    }
    issue_tile<SEFF, FP4>(e, piece, ring_s + s * kSlot, bar_s + 8 * s, lane);
    issued++;
  };
  for (int i = 0; i < kRing<FP4>; i++) produce();

  // q of the unit: rotated and cut by all warps.
  if (tid < G * kD / 8) reinterpret_cast<uint4*>(qraw)[tid] = qv;
  __syncthreads();
  prep_q<G, kWarps, FP4>(qraw, frag, sf, lane, p, w);
  __syncthreads();
  typename QF<G, FP4>::type qf;
  qfrag_get<G>(qf, frag, sf, lane);

  State<G> st;
  state_reset<G>(st);
  constexpr int NQ = QFrag<G>::NQ;
  float sc[2][NQ][2], alpha[NQ];
  int consumed = 0, slot_i = 0;
  uint32_t parity = 0;
  bool dead = false;
  auto valid_of = [&](int s) {
    // (the form that suits the format, as in the decode kernel; two pages need a prefix each)
    const int2 v = valid_ring[w][s];
    if constexpr (FP4 && kPPT == 1) return v.x;
    else return Valid{{v.x, v.y}};
  };
  if (issued > 0) {
    if (!mbar_wait_warp(bar_s, 0u, kWaitLimitNs)) {
      dead = true;
    } else {
      tile_qk_any<G, SEFF>(qf, ring_w, valid_of(0), lane, sc);
      if (tile_softmax_stats<G>(st, sc, alpha)) tile_rescale<G>(st, alpha);
    }
  }
  // As in the decode kernel: the scores and statistics of the next tile next to the PV of the
  // current one.
  while (consumed + 1 < issued && !dead) {
    const int cs = slot_i, ns = cs + 1 == kRing<FP4> ? 0 : cs + 1;
    const uint32_t npar = cs + 1 == kRing<FP4> ? parity ^ 1u : parity;
    if (!mbar_wait_warp(bar_s + 8 * ns, npar, kWaitLimitNs)) {
      dead = true;
      break;
    }
    float sn[2][NQ][2];
    tile_qk_any<G, SEFF>(qf, ring_w + ns * kSlot, valid_of(ns), lane, sn);
    const bool rescale = tile_softmax_stats<G>(st, sn, alpha);
    tile_pv_any<G, SEFF, FP4>(st, ring_w + cs * kSlot, valid_of(cs), lane, sc);
    consumed++;
    slot_i = ns;
    parity = npar;
    __syncwarp();
    fence_proxy_async_smem();
    produce();
    if (rescale) tile_rescale<G>(st, alpha);
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int qq = 0; qq < NQ; qq++)
#pragma unroll
        for (int r = 0; r < 2; r++) sc[j][qq][r] = sn[j][qq][r];
  }
  if (issued > 0 && !dead) {
    tile_pv_any<G, SEFF, FP4>(st, ring_w + slot_i * kSlot, valid_of(slot_i), lane, sc);
    consumed++;
  }
  if (dead) {
    // Flag it and let the copies still in flight land (bounded) before their memory is reused.
    if (lane == 0) atomicOr(p.status, KVQ_DEV_TIMEOUT_BIT);
    for (int j = consumed; j < issued; j++)
      mbar_wait_warp(bar_s + 8 * (j % kRing<FP4>), static_cast<uint32_t>((j / kRing<FP4>) & 1), kWaitLimitNs);
  }
  // The warps' records, each in its own drained ring; an idle warp's has m = -inf, l = 0.
  __syncwarp();
  float* const rec_w = reinterpret_cast<float*>(ring_w);
  state_write<G>(st, rec_w, lane);
  __syncthreads();
  __half* const orow = p.out + (static_cast<size_t>(t) * p.num_kv_heads + h) * G * kD;
  auto rec = [&](int j) -> const float* { return reinterpret_cast<const float*>(ring) + j * (kRing<FP4> * kSlot / 4); };
  auto part_rec = [&](int j) { return p.part + (static_cast<size_t>(unit) * splits + j) * G * kPartStride; };
  merge_few<G, kWarps, false, kWarps>(kWarps, rec, w, orow, splits > 1 ? part_rec(part) : nullptr, lane, p);
  if (splits == 1) return;
  __syncthreads();
  if (tid == 0) {
    const int old = atom_add_acq_rel_gpu(p.counters + unit, 1);
    last_flag = old == splits - 1;
    if (last_flag) p.counters[unit] = 0;  // ready for the next call
  }
  __syncthreads();
  if (!last_flag) return;
  merge_few<G, kWarps, true, kMaxSplits>(splits, [&](int j) -> const float* { return part_rec(j); }, w, orow, nullptr,
                                         lane, p);
}

size_t smem_bytes(int group, bool fp4) {
  size_t s = static_cast<size_t>(kWarps) * (fp4 ? kRing<true> : kRing<false>) * slot_bytes(fp4);
  s += static_cast<size_t>(group) * kD * 2 + sizeof(uint32_t) * frag_words(group, fp4) + 8 * sizeof(float);
  s += sizeof(uint64_t) * kWarps * 4 + 128;
  return (s + 15) & ~static_cast<size_t>(15);
}

template <int G, int SEFF, bool FP4>
int launch_one(const cudaLaunchConfig_t& cfg, const DecodeParams& p, const SparseParams& sp, int splits) {
  if (!ensure_smem<sparse_kernel<G, SEFF, FP4>>(smem_bytes(G, FP4))) return -2;
  return cudaLaunchKernelEx(&cfg, sparse_kernel<G, SEFF, FP4>, p, sp, splits) == cudaSuccess ? 0 : -2;
}

template <int G>
int launch_group(const cudaLaunchConfig_t& cfg, const DecodeParams& p, const SparseParams& sp, int splits) {
  if (p.page_size < kTileTokens)
    return p.fp4 ? launch_one<G, 16, true>(cfg, p, sp, splits) : launch_one<G, 16, false>(cfg, p, sp, splits);
  return p.fp4 ? launch_one<G, 32, true>(cfg, p, sp, splits) : launch_one<G, 32, false>(cfg, p, sp, splits);
}

}  // namespace

int launch_sparse(const DecodeParams& p, const SparseParams& sp, int num_sms, cudaStream_t stream) {
  const long long units = static_cast<long long>(sp.total_q) * p.num_kv_heads;
  if (units == 0) return 0;
  // Parts of a unit: as many as fill the SMs' CTAs, while every warp keeps a tile and
  // the scratch has a record and a counter for each.
  const int ntile = static_cast<int>((static_cast<long long>(sp.num_blocks) * p.page_size + kTileTokens - 1) / kTileTokens);
  int splits = 1;
  if (units <= sp.num_counters) {
    const long long fit = static_cast<long long>(kCtasPerSm) * num_sms / units, slots = sp.num_slots / units, work = (ntile + kWarps - 1) / kWarps;
    long long s = fit < kMaxSplits ? fit : kMaxSplits;
    if (s > slots) s = slots;
    if (s > work) s = work;
    if (s > 1) splits = static_cast<int>(s);
  }
  if (units * splits > 0x7fffffffLL) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(p.group, p.fp4 != 0);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (p.group) {
    case 1: return launch_group<1>(cfg, p, sp, splits);
    case 2: return launch_group<2>(cfg, p, sp, splits);
    case 4: return launch_group<4>(cfg, p, sp, splits);
    case 8: return launch_group<8>(cfg, p, sp, splits);
    default: return -1;
  }
}

}  // namespace kvq
