// decode_kernel.cu -- paged GQA decode attention over the rotated INT4 cache, sm_100a.
//
// Method: "KVキャッシュを4ビットへ — SAW-INT4とシステムを踏まえたINT4量子化"
// (youngju.dev), section "KVキャッシュこそが本当のボトルネックである理由" (paged memory
// layout, regular access, fused attention execution) and section "回転のトリック —
// ブロック対角アダマール" (the rotation is orthogonal, so q.k is unchanged when both are
// rotated, and the rotation is undone exactly on the output).  Every decode step streams
// the whole cache, so the kernel is HBM-bound; everything below serves keeping the bytes
// moving with few instructions per byte.
//
// Work split (one launch).  The cache is cut into tiles of 32 tokens of one (sequence,
// KV head) "unit", numbered unit-major.  CTA k takes the contiguous tile range
// [k*chunk, (k+1)*chunk) of the T tiles, chunk = ceil(T/C), so every CTA streams the
// same number of bytes whatever the length mix.  Its 4 warps take the range's tiles in
// turn (tile X0 + w, X0 + w + 4, ...), each keeping an online-softmax state per unit; at
// the end of each unit the warps merge through shared memory.  A unit inside one CTA is finished
// there (normalise, inverse rotation, fp16 store).  A unit spanning several CTAs leaves
// one (o', m, l) partial per CTA in scratch slot unit + k (unique along the staircase of
// ranges); the last CTA to arrive (an atomic counter per unit, reset after use) merges
// them and finishes the unit.  The rotated, sliced q of a unit is prepared once per CTA
// (warp w takes query w) into a shared table the warps load their fragments from.
//
// Loads.  Each warp owns a ring of 3 shared-memory slots of one tile each.  Per tile one
// lane per page issues a 1-D bulk copy (cp.async.bulk, TMA engine, no multicast) of the
// contiguous (page, head) block -- codes and scales together -- into a slot, completing
// on the slot's mbarrier.  Page ids are read in batches, one per lane, a batch ahead of
// use, and sequence lengths are kept in shared memory, so no global-memory latency sits
// between consuming a tile and issuing the copy that refills its slot.
//
// QK^T on tensor cores in exact integer arithmetic: mma.sync m16n8k32 s8 x s8 -> s32 with
// A = K codes (16 tokens x 32 channels) and B = the rotated, scaled q cut into three int8
// slices, q' = M/64 * (q1 + q2/128 + q3/16384) with M the power of two above max|q'| (so
// q' is carried to 2^-21 of M).  A nibble becomes an int8 of value 16n with one or two
// bit operations (shift the nibble to the byte's top).  The channel order inside each
// k32 step is chosen so that a thread's fragment is one 32-bit word of codes (a dot
// product does not depend on the order of its terms).
// PV on tensor cores: mma.sync m16n8k16 f16 x f16 -> f32 with A = V codes transposed
// (16 channels x 16 tokens, gathered with byte permutes, exact fp16 integers) and B = P'
// = p * s_v (the V scale folded into the probabilities) as fp16 hi + lo parts: for G <= 4
// the two parts sit in neighbouring columns, for G = 8 two MMAs accumulate them.  (The
// integer values go in exactly, without a constant offset: the tensor core's internal
// sum is not precise enough to cancel a large offset afterwards.)  The GQA group is the N = 8
// side of both products; the dequantised cache is the M side.  The K scale multiplies the
// fp32 score of its token; softmax runs in the log2 domain with exp2.
//
// NVFP4 cache (template argument FP4; "BitDecoding-FP4:FP4 KVキャッシュのネイティブ復号"
// (sns.style): E2M1 codes with an E4M3 scale per 16 channels, 144-byte token rows): the
// same work split, rings and merges; K and V are dequantised exactly to fp16 (hardware
// E2M1 / E4M3 conversions and one fp16 multiply), both products run as f16 mma.sync, and q
// is carried as fp16 hi + lo parts (tile_qk4, tile_pv4, prep_q4_warp).
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include "decode_tile.cuh"
#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

namespace {

__device__ __forceinline__ int clamp_len(int L, int cap, int32_t* status) {
  if (L < 0 || L > cap) {
    atomicOr(status, KVQ_DEV_BAD_POS_BIT);
    return L < 0 ? 0 : cap;
  }
  return L;
}

// One (sequence, KV head) unit and its place in the tile sequence.  pre[] (tiles per
// sequence, exclusive prefix) and lens[] (clamped lengths) live in shared memory.
struct Unit {
  int b, h;  // sequence, KV head
  int n;     // tiles in the unit
  int L;     // tokens
  int U;     // global index of the unit's first tile
};

__device__ __forceinline__ void unit_of_tile(Unit& u, int x, const int32_t* pre, const int32_t* lens,
                                             const DecodeParams& p) {
  int lo = 0, hi = p.batch;  // pre[lo]*Hkv <= x < pre[hi]*Hkv
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * p.num_kv_heads <= x) lo = mid; else hi = mid;
  }
  u.b = lo;
  u.n = pre[lo + 1] - pre[lo];
  const int base = pre[lo] * p.num_kv_heads;
  u.h = (x - base) / u.n;
  u.U = base + u.h * u.n;
  u.L = lens[lo];
}

// The next non-empty unit.  Callers only ask while one exists.
__device__ __forceinline__ void unit_next(Unit& u, const int32_t* pre, const int32_t* lens,
                                          const DecodeParams& p) {
  if (++u.h == p.num_kv_heads) {
    u.h = 0;
    do { ++u.b; } while (u.b < p.batch && pre[u.b + 1] == pre[u.b]);
    if (u.b >= p.batch) return;
    u.n = pre[u.b + 1] - pre[u.b];
    u.L = lens[u.b];
  }
  u.U = pre[u.b] * p.num_kv_heads + u.h * u.n;
}

// ------------------------------------------------------------------- copies --
// Page entries of a warp's upcoming tiles, one per lane: a batch covers kBatch tiles of
// kPPT pages (tile t of the warp = CTA tile X0 + w + kWarps*t).  Entry lane: tile
// tb + lane / kPPT, page lane % kPPT of the tile, as the address of that (page, head)
// block with flags in its low 4 bits (blocks are 16-byte aligned): bits 0-2 = the
// tile's first token in the page / 32 (pages of 64+ tokens), bit 3 = the page id was out
// of range (page 0 is read instead and the status word is flagged at issue); 0 where no
// page is needed.
template <int SEFF>
struct PageBatch {
  static constexpr int kPPT = (SEFF < kTileTokens) ? kTileTokens / SEFF : 1;
  static constexpr int kBatch = 32 / kPPT;
};

constexpr uint64_t kEntryBad = 8u;

template <int SEFF, bool FP4>
__device__ __forceinline__ uint64_t load_page_batch(int tb, int X0, int X1, int w, int lane,
                                                    const int32_t* pre, const int32_t* lens,
                                                    const DecodeParams& p) {
  constexpr int kPPT = PageBatch<SEFF>::kPPT;
  const int x = X0 + w + kWarps * (tb + lane / kPPT);
  uint64_t e = 0;
  if (x < X1) {
    Unit u;
    unit_of_tile(u, x, pre, lens, p);
    const int t0 = (x - u.U) * kTileTokens;
    const int lp = (t0 >> p.page_shift) + lane % kPPT;
    if ((lp << p.page_shift) < u.L) {
      int pid = __ldg(p.page_table + static_cast<size_t>(u.b) * p.max_pages_per_seq + lp);
      uint64_t flags = 0;
      if (pid < 0 || pid >= p.num_pages) {
        pid = 0;
        flags = kEntryBad;
      }
      const size_t blk_bytes = static_cast<size_t>(p.page_size) * row_bytes(FP4);
      e = reinterpret_cast<uint64_t>(p.pool_layer +
                                     (static_cast<size_t>(pid) * p.num_kv_heads + u.h) * blk_bytes);
      if (SEFF == kTileTokens) e |= static_cast<uint64_t>((t0 & (p.page_size - 1)) / kTileTokens);
      e |= flags;
    }
  }
  return e;
}

// Issue the bulk copies of one tile into a ring slot (the whole warp calls; lane j <
// kPPT holds the tile's page entry j).  The slot holds a virtual page of SEFF = min(S, 32)
// token slots per copied page, [K codes][V codes][K scales][V scales], the pool's own
// block layout.
template <int SEFF, bool FP4>
__device__ __forceinline__ void tile_issue(uint64_t e, uint32_t slot, uint32_t bar, int lane,
                                           uint64_t pol, const DecodeParams& p) {
  constexpr int kPPT = PageBatch<SEFF>::kPPT;
  const bool have = lane < kPPT && e != 0;
  if (__any_sync(kFull, have && (e & kEntryBad)) && lane == 0) atomicOr(p.status, KVQ_DEV_BAD_PAGE_BIT);
  const int S = p.page_size;
  if (SEFF < kTileTokens || S == kTileTokens) {
    const uint8_t* blk = reinterpret_cast<const uint8_t*>(e & ~static_cast<uint64_t>(15));
    const uint32_t blk_bytes = static_cast<uint32_t>(S) * row_bytes(FP4);
    const int npg = __popc(__ballot_sync(kFull, have));
    if (lane == 0) mbar_arrive_expect_tx(bar, npg * blk_bytes);
    __syncwarp();
    if (have) bulk_copy_g2s(slot + lane * blk_bytes, blk, blk_bytes, bar, pol);
  } else {
    // One page per tile; lanes 0-3 copy its K codes, V codes, K scales and V scales.
    const uint64_t e0 = __shfl_sync(kFull, e, 0);
    const uint8_t* blk = reinterpret_cast<const uint8_t*>(e0 & ~static_cast<uint64_t>(15));
    const size_t o = static_cast<size_t>(e0 & 7u) * kTileTokens;  // tile's first token in the page
    const uint8_t* src = blk + o * 64;
    uint32_t dst = slot, bytes = 2048;
    if constexpr (FP4) {  // scales: 8 E4M3 bytes per token row
      if (lane == 1) { src = blk + static_cast<size_t>(S) * 64 + o * 64; dst = slot + 2048; }
      if (lane == 2) { src = blk + static_cast<size_t>(S) * 128 + o * 8; dst = slot + 4096; bytes = 256; }
      if (lane == 3) { src = blk + static_cast<size_t>(S) * 136 + o * 8; dst = slot + 4352; bytes = 256; }
    } else {
      if (lane == 1) { src = blk + static_cast<size_t>(S) * 64 + o * 64; dst = slot + 2048; }
      if (lane == 2) { src = blk + static_cast<size_t>(S) * 128 + o * 2; dst = slot + 4096; bytes = 64; }
      if (lane == 3) { src = blk + static_cast<size_t>(S) * 130 + o * 2; dst = slot + 4160; bytes = 64; }
    }
    if (lane == 0) mbar_arrive_expect_tx(bar, slot_bytes(FP4));
    __syncwarp();
    if (lane < 4) bulk_copy_g2s(dst, src, bytes, bar, pol);
  }
}

// A warp's producer: issues its tiles t = 0, 1, ... (CTA tile X0 + w + kWarps*t) in
// order into its ring, slot t % kStages; page entries come from batches loaded one
// batch ahead.
template <int SEFF, bool FP4>
struct Producer {
  int t;         // next tile to issue
  int nT;        // tiles of this warp
  int tb;        // first tile of the current batch
  uint64_t cur;  // this lane's entry of the current batch
  uint64_t nxt;  // ... of the next batch
};

template <int SEFF, bool FP4>
__device__ __forceinline__ void producer_issue(Producer<SEFF, FP4>& pr, int X0, int X1, int w, int lane,
                                               uint32_t ring_s, uint32_t bar_s, uint64_t pol,
                                               const int32_t* pre, const int32_t* lens,
                                               const DecodeParams& p) {
  constexpr int kPPT = PageBatch<SEFF>::kPPT, kBatch = PageBatch<SEFF>::kBatch;
  if (pr.t >= pr.tb + kBatch) {
    pr.tb += kBatch;
    pr.cur = pr.nxt;
    pr.nxt = pr.tb + kBatch < pr.nT ? load_page_batch<SEFF, FP4>(pr.tb + kBatch, X0, X1, w, lane, pre, lens, p) : 0;
  }
  const int src = (pr.t - pr.tb) * kPPT + lane;
  const uint64_t e = __shfl_sync(kFull, pr.cur, src & 31);
  const int s = pr.t % kStages;
  tile_issue<SEFF, FP4>(e, ring_s + s * slot_bytes(FP4), bar_s + 8 * s, lane, pol, p);
  pr.t++;
}

// Merge nrec partial records of one unit (record j: [G][kPartStride] floats at rec(j)) for
// the queries q0, q0 + QSTEP, ... < G (one warp; lane: channels 4*lane..4*lane+3), then
// either finish them into orow or, with crec != nullptr, store the merged record there.
// Records are taken 32 at a time with an online rescale: lane j fetches (m, l) of record j
// of the chunk for every owned query, in the same round as the o' rows of the chunk's
// first records (8 float4 per lane a round), so a merge of a few records costs one round
// trip to L2.
// GLOBAL: the records were written by other warps or CTAs and are read from L2.
template <int G, int QSTEP, bool GLOBAL, typename F>
__device__ __forceinline__ void merge_records(int nrec, F&& rec, int q0, __half* orow, float* crec,
                                              int lane, const DecodeParams& p) {
  constexpr int NQW = (G + QSTEP - 1) / QSTEP;       // queries this warp handles (at most)
  constexpr int R = (8 / NQW) < 1 ? 1 : 8 / NQW;     // records per round of o' loads
  if (q0 >= G) return;
  float M[NQW], l[NQW], o[NQW][4];
#pragma unroll
  for (int i = 0; i < NQW; i++) {
    M[i] = -CUDART_INF_F;
    l[i] = 0.0f;
    o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
  }
  for (int base = 0; base < nrec; base += 32) {
    const bool mine = base + lane < nrec;
    const float* rj = mine ? rec(base + lane) : nullptr;
    const int cnt = min(32, nrec - base);
    // o' rows of records base .. base + R - 1, fetched together with the (m, l) pairs.
    float4 v[R][NQW];
    auto fetch = [&](int j0) {
#pragma unroll
      for (int r = 0; r < R; r++) {
        const int j = j0 + r;
        const float* rr = (j < cnt) ? rec(base + j) : nullptr;
#pragma unroll
        for (int i = 0; i < NQW; i++) {
          const int qi = min(q0 + i * QSTEP, G - 1);
          v[r][i] = rr ? ld_rec4<GLOBAL>(rr + qi * kPartStride + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    };
    fetch(0);
    float e[NQW];
    float2 ml[NQW];
#pragma unroll
    for (int i = 0; i < NQW; i++) {
      const int qi = min(q0 + i * QSTEP, G - 1);
      ml[i] = mine ? ld_rec2<GLOBAL>(rj + qi * kPartStride + kD) : make_float2(-CUDART_INF_F, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < NQW; i++) {
      float mc = ml[i].x;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mc = fmaxf(mc, __shfl_xor_sync(kFull, mc, d));
      const float Mn = fmaxf(M[i], mc);  // finite: every record holds at least one token
      const float r = (M[i] == -CUDART_INF_F) ? 0.0f : exp2f(M[i] - Mn);
      M[i] = Mn;
      l[i] *= r;
#pragma unroll
      for (int c = 0; c < 4; c++) o[i][c] *= r;
      e[i] = (ml[i].x == -CUDART_INF_F) ? 0.0f : exp2f(ml[i].x - Mn);
      float le = e[i] * ml[i].y;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) le += __shfl_xor_sync(kFull, le, d);
      l[i] += le;
    }
    for (int j0 = 0; j0 < cnt; j0 += R) {
      if (j0 > 0) fetch(j0);
#pragma unroll
      for (int r = 0; r < R; r++) {
#pragma unroll
        for (int i = 0; i < NQW; i++) {
          const float ej = __shfl_sync(kFull, e[i], (j0 + r) & 31);  // 0 past cnt: v is 0 too
          o[i][0] += ej * v[r][i].x;
          o[i][1] += ej * v[r][i].y;
          o[i][2] += ej * v[r][i].z;
          o[i][3] += ej * v[r][i].w;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NQW; i++) {
    const int qi = q0 + i * QSTEP;
    if (qi >= G) continue;
    if (crec) {
      float* r = crec + qi * kPartStride;
      *reinterpret_cast<float4*>(r + 4 * lane) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
      if (lane == 0) *reinterpret_cast<float2*>(r + kD) = make_float2(M[i], l[i]);
    } else {
      finish_query(o[i], l[i], orow + qi * kD, lane, p);
    }
  }
}

// --------------------------------------------------------- fused append --
// One new token of one (sequence, KV head): its K or V row rotated and quantised by a
// warp, bit-identical to the append kernel (the fixed-order butterfly: stages h = 1, 2
// inside a lane's 4 channels, h = 4..64 across lanes as fma(own, +-1, other), one rounding
// each; then y = fl(y * c_b); s = fp16(fl(max|y| / 7)); codes = round-half-even of y / s
// decided exactly by comparing y with (k + 1/2) * s, clamped to [-8, 7]).  Lane L gets the
// 16 code bits of channels 4L..4L+3 (low nibble = even channel) and the fp16 scale bits.
struct NewRow {
  uint32_t codes16;  // this lane's 2 bytes of the packed row
  uint32_t scale;    // fp16 bits, same in every lane
};

// Channels 4*lane..4*lane+3 of a row that another kernel may still be writing (a load before
// the wait): each word is one that was there, and a later load is not served from this one's line.
__device__ __forceinline__ uint2 load_new_row(const __half* row, int lane) {
  uint2 r;
  asm volatile("ld.relaxed.gpu.global.v2.u32 {%0,%1}, [%2];"
               : "=r"(r.x), "=r"(r.y)
               : "l"(reinterpret_cast<const uint2*>(row) + lane)
               : "memory");
  return r;
}

// The rotated row y = fl(c_b * butterfly(x)) of channels 4*lane..4*lane+3.
__device__ __forceinline__ void rotate_new_row(uint2 raw, int lane, const DecodeParams& p, float (&x)[4]) {
  const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
  const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
  x[0] = lo.x;
  x[1] = lo.y;
  x[2] = hi.x;
  x[3] = hi.y;
  if (p.hadamard_block > 1) {
    const float a0 = __fadd_rn(x[0], x[1]), a1 = __fsub_rn(x[0], x[1]);
    const float a2 = __fadd_rn(x[2], x[3]), a3 = __fsub_rn(x[2], x[3]);
    x[0] = __fadd_rn(a0, a2);
    x[2] = __fsub_rn(a0, a2);
    x[1] = __fadd_rn(a1, a3);
    x[3] = __fsub_rn(a1, a3);
#pragma unroll
    for (int st = 0; st < 5; st++) {
      if ((4 << st) < p.hadamard_block) {
        const float sgn = ((lane >> st) & 1) ? -1.0f : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = __fmaf_rn(x[e], sgn, __shfl_xor_sync(kFull, x[e], 1 << st));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; e++) x[e] = __fmul_rn(x[e], p.cb);
  }
}

__device__ __forceinline__ NewRow quantise_new_row(uint2 raw, int lane, const DecodeParams& p) {
  float x[4];
  rotate_new_row(raw, lane, p, x);
  float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
  for (int d = 1; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
  const float s32 = __fdiv_rn(m, 7.0f);
  const __half sh = s32 > 65504.0f ? __ushort_as_half(0x7BFF) : __float2half_rn(s32);
  const float s = __half2float(sh);
  NewRow r;
  r.scale = __half_as_ushort(sh);
  r.codes16 = 0u;
  if (s != 0.0f) {
    const float rc = __frcp_rn(s), hs = 0.5f * s;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const float k = floorf(__fmul_rn(x[e], rc));
      const float h = __fmaf_rn(k, s, hs);  // (k + 1/2) * s, exact
      const bool odd = (__float_as_uint(__fadd_rn(k, kMagic)) & 1u) != 0u;
      const bool up = x[e] > h || (x[e] == h && odd);
      const int c = static_cast<int>(fminf(fmaxf(up ? k + 1.0f : k, -8.0f), 7.0f));
      r.codes16 |= (static_cast<uint32_t>(c) & 0xFu) << (4 * e);
    }
  }
  return r;
}

// NVFP4 new row, bit-identical to the append kernel: lanes 4m..4m+3 hold block m (16
// channels); s = E4M3(fl(max |y| / 6)) (nearest even, saturating), codes = E2M1(fl(y *
// fl(1/s))) (nearest even, saturating, sign kept), 0 when s == 0.  codes16 = the lane's two
// code bytes; scale = block m's E4M3 byte (the same in its 4 lanes).
__device__ __forceinline__ NewRow quantise_new_row_fp4(uint2 raw, int lane, const DecodeParams& p) {
  float x[4];
  rotate_new_row(raw, lane, p, x);
  float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
  m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
  m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
  uint16_t sb2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb2) : "f"(0.0f), "f"(__fdiv_rn(m, 6.0f)));
  const uint32_t sh = e4m3x2_to_f16x2(sb2);
  const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(sh & 0xFFFFu)));
  NewRow r;
  r.scale = sb2 & 0xFFu;
  r.codes16 = 0u;
  if (s != 0.0f) {
    const float rc = __frcp_rn(s);
    uint32_t b0, b1;
    asm("{\n\t.reg .b8 q;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %1, %2;\n\tcvt.u32.u8 %0, q;\n\t}"
        : "=r"(b0) : "f"(__fmul_rn(x[1], rc)), "f"(__fmul_rn(x[0], rc)));
    asm("{\n\t.reg .b8 q;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %1, %2;\n\tcvt.u32.u8 %0, q;\n\t}"
        : "=r"(b1) : "f"(__fmul_rn(x[3], rc)), "f"(__fmul_rn(x[2], rc)));
    r.codes16 = b0 | (b1 << 8);
  }
  return r;
}

// Bytes of a token's scales in a block row (K, then V) and the patch buffer's layout:
// [K codes 64 B][V codes 64 B][K scales][V scales], then the token's place in its tile.
template <bool FP4>
struct PatchLayout {
  static constexpr int kScale = FP4 ? kD / 16 : 2;   // per K or V row
  static constexpr int kJ = 128 + 2 * kScale;          // 132 or 144
};

// The new token of a unit (its raw K and V rows kraw, vraw as loaded by load_new_row):
// rotate and quantise the rows into the warp's patch buffer (shared memory), in the block
// layout of one token.
template <bool FP4>
__device__ __forceinline__ void fused_quantise(uint2 kraw, uint2 vraw, int lane, uint8_t* patch,
                                               const DecodeParams& p) {
  if constexpr (FP4) {
    const NewRow kr = quantise_new_row_fp4(kraw, lane, p);
    const NewRow vr = quantise_new_row_fp4(vraw, lane, p);
    *reinterpret_cast<uint16_t*>(patch + 2 * lane) = static_cast<uint16_t>(kr.codes16);
    *reinterpret_cast<uint16_t*>(patch + 64 + 2 * lane) = static_cast<uint16_t>(vr.codes16);
    if ((lane & 3) == 0) {
      patch[128 + (lane >> 2)] = static_cast<uint8_t>(kr.scale);
      patch[136 + (lane >> 2)] = static_cast<uint8_t>(vr.scale);
    }
  } else {
    const NewRow kr = quantise_new_row(kraw, lane, p);
    const NewRow vr = quantise_new_row(vraw, lane, p);
    *reinterpret_cast<uint16_t*>(patch + 2 * lane) = static_cast<uint16_t>(kr.codes16);
    *reinterpret_cast<uint16_t*>(patch + 64 + 2 * lane) = static_cast<uint16_t>(vr.codes16);
    if (lane == 0) {
      *reinterpret_cast<uint16_t*>(patch + 128) = static_cast<uint16_t>(kr.scale);
      *reinterpret_cast<uint16_t*>(patch + 130) = static_cast<uint16_t>(vr.scale);
    }
  }
  __syncwarp();
}

// Store the patch buffer's token of unit (b, h) at position seq_lens[b] of the pool
// (skipped, with the status flagged, when the position or its page is out of range).
// Returns whether it is stored and belongs in the decode.
template <bool FP4>
__device__ __forceinline__ bool fused_store(int b, int h, int lane, const uint8_t* patch,
                                            const DecodeParams& p) {
  constexpr int SC = PatchLayout<FP4>::kScale;
  const int pos = __ldg(p.seq_lens + b);
  const int S = p.page_size;
  const int lp = pos >> p.page_shift;
  if (pos < 0 || lp >= p.max_pages_per_seq) return false;  // flagged by the length clamp
  const int page = __ldg(p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq + lp);
  if (page < 0 || page >= p.num_pages) return false;     // flagged when the tile is issued
  const int slot = pos & (S - 1);
  uint8_t* blk = const_cast<uint8_t*>(p.pool_layer) + (static_cast<size_t>(page) * p.num_kv_heads + h) *
                                      (static_cast<size_t>(S) * (kD + 2 * SC));
  const uint16_t kc = *reinterpret_cast<const uint16_t*>(patch + 2 * lane);
  const uint16_t vc = *reinterpret_cast<const uint16_t*>(patch + 64 + 2 * lane);
  *reinterpret_cast<uint16_t*>(blk + slot * 64 + 2 * lane) = kc;
  *reinterpret_cast<uint16_t*>(blk + S * 64 + slot * 64 + 2 * lane) = vc;
  if (lane == 0) {
    if constexpr (FP4) {
      *reinterpret_cast<uint2*>(blk + S * 128 + slot * 8) = *reinterpret_cast<const uint2*>(patch + 128);
      *reinterpret_cast<uint2*>(blk + S * 136 + slot * 8) = *reinterpret_cast<const uint2*>(patch + 136);
    } else {
      *reinterpret_cast<uint16_t*>(blk + S * 128 + slot * 2) = *reinterpret_cast<const uint16_t*>(patch + 128);
      *reinterpret_cast<uint16_t*>(blk + S * 130 + slot * 2) = *reinterpret_cast<const uint16_t*>(patch + 130);
    }
  }
  return true;
}

// Overwrite token j (0..31, kept at byte PatchLayout::kJ of the patch buffer) of a landed
// ring slot with the patch buffer's token (the slot's copy of the pool may predate the
// store above).  The warp syncs before the slot is read.
template <int SEFF, bool FP4>
__device__ __forceinline__ void patch_slot(uint8_t* slot, int lane, const uint8_t* patch) {
  constexpr int SC = PatchLayout<FP4>::kScale;
  const int j = *reinterpret_cast<const int*>(patch + PatchLayout<FP4>::kJ);  // place in the tile
  uint8_t* base = slot + (j / SEFF) * (SEFF * row_bytes(FP4));
  const int jj = j % SEFF;
  const uint32_t wv = reinterpret_cast<const uint32_t*>(patch)[lane];  // bytes 4*lane..
  uint8_t* dst = lane < 16 ? base + jj * 64 + 4 * lane : base + SEFF * 64 + jj * 64 + 4 * (lane - 16);
  *reinterpret_cast<uint32_t*>(dst) = wv;
  if (lane == 0) {
    if constexpr (FP4) {
      *reinterpret_cast<uint2*>(base + SEFF * 128 + jj * SC) = *reinterpret_cast<const uint2*>(patch + 128);
      *reinterpret_cast<uint2*>(base + SEFF * (128 + SC) + jj * SC) = *reinterpret_cast<const uint2*>(patch + 136);
    } else {
      *reinterpret_cast<uint16_t*>(base + SEFF * 128 + jj * 2) = *reinterpret_cast<const uint16_t*>(patch + 128);
      *reinterpret_cast<uint16_t*>(base + SEFF * 130 + jj * 2) = *reinterpret_cast<const uint16_t*>(patch + 130);
    }
  }
  __syncwarp();
}

// FUSED: the one-token append runs inside (p.k_new, p.v_new set).
// FP4: the cache holds NVFP4 rows.
template <int G, int SEFF, bool FUSED, bool FP4>
__global__ void __launch_bounds__(kThreads, 3) decode_kernel(DecodeParams p) {
  constexpr int kFragWords = frag_words(G, FP4);
  constexpr int kSlot = slot_bytes(FP4);
  extern __shared__ __align__(128) uint8_t smem_raw[];
  // Bulk copies need 16-byte aligned destinations; align to 128 bytes (the allocation
  // carries 128 spare bytes for this).
  uint8_t* smem = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
  uint8_t* ring = smem;                                                      // [w][stage][4224]
  // Per warp (index w) and two more for the CTA's first and last unit (indices kWarps,
  // kWarps + 1): raw q rows, fragment table, M factors.
  constexpr int kQT = kWarps + 2;
  uint8_t* qraw_all = ring + kWarps * kStages * kSlot;                       // [kQT][G][128] fp16
  uint32_t* frag_all = reinterpret_cast<uint32_t*>(qraw_all + kQT * G * kD * 2);  // [kQT][kFragWords]
  float* sf_all = reinterpret_cast<float*>(frag_all + kQT * kFragWords);     // [kQT][8]
  float* mbuf = sf_all + kQT * 8;                                            // [w][G][132]
  uint64_t* bars = reinterpret_cast<uint64_t*>(mbuf + kWarps * G * kPartStride);  // [w][kStages+1], CTA q
  int32_t* pre = reinterpret_cast<int32_t*>(bars + kWarps * (kStages + 1) + 1);  // [batch + 1]
  int32_t* lens = pre + p.batch + 1;                                         // [batch]
  __shared__ int warp_sum[kWarps];
  __shared__ int running;
  __shared__ int last_flag_e[2];

  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int cap = p.max_pages_per_seq * p.page_size;
  // The prologue below reads only seq_lens and the page table, which no kernel of this
  // library writes (and may OR bits into the status word); everything else an earlier
  // kernel may write or read (pool, q, out, the scratch) is touched only after
  // griddep_wait(), and the new K/V rows are what they are after it.
  griddep_launch_dependents();

  const uint32_t qbar_cta = smem_addr(bars + kWarps * (kStages + 1));
  if (tid == 0) {
    mbar_init(qbar_cta, 1);
    fence_mbar_init();
  }

  // Clamped lengths, and tiles per sequence -> exclusive prefix pre[0..batch].
  if (tid == 0) running = 0;
  __syncthreads();
  for (int base = 0; base < p.batch; base += kThreads) {
    const int i = base + tid;
    int n = 0;
    if (i < p.batch) {
      const int L = clamp_len(__ldg(p.seq_lens + i) + (FUSED ? 1 : 0), cap, p.status);
      lens[i] = L;
      n = (L + kTileTokens - 1) / kTileTokens;
    }
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int y = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += y;
    }
    if (lane == 31) warp_sum[w] = incl;
    __syncthreads();
    int before = running;
    for (int w2 = 0; w2 < w; w2++) before += warp_sum[w2];
    if (i < p.batch) pre[i] = before + incl - n;
    __syncthreads();
    if (tid == kThreads - 1) running = before + incl;
    __syncthreads();
  }
  if (tid == 0) pre[p.batch] = running;
  __syncthreads();

  // CTA k takes tiles [k*chunk, (k+1)*chunk) of the T tiles (the host bounds T < 2^30);
  // warp w of it takes tiles X0 + w, X0 + w + kWarps, ...
  const int T = pre[p.batch] * p.num_kv_heads;
  const int chunk = (T + p.total_ctas - 1) / p.total_ctas;
  const int kc = blockIdx.x;
  const int X0 = kc * chunk;
  const int X1 = min(T, X0 + chunk);
  const bool has_tiles = T > 0 && X0 < T;

  uint8_t* qraw = qraw_all + w * G * kD * 2;
  uint32_t* frag = frag_all + w * kFragWords;
  float* sf = sf_all + w * 8;
  uint8_t* ring_w = ring + w * kStages * kSlot;
  const uint8_t* ring_p = ring_w;
  const uint32_t ring_s = smem_addr(ring_p);
  const uint32_t bar_s = smem_addr(bars + w * (kStages + 1));
  const uint32_t qbar = bar_s + 8 * kStages;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s <= kStages; s++) mbar_init(bar_s + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();
  const uint64_t pol = l2_policy_evict_first();

  // Producer: page-id batches 0 and 1 (page table only: before the wait).
  constexpr int kBatch = PageBatch<SEFF>::kBatch;
  Producer<SEFF, FP4> pr;
  pr.t = 0;
  pr.nT = has_tiles ? max(0, (X1 - X0 - w + kWarps - 1) / kWarps) : 0;
  pr.tb = 0;
  pr.cur = has_tiles ? load_page_batch<SEFF, FP4>(0, X0, X1, w, lane, pre, lens, p) : 0;
  pr.nxt = pr.nT > kBatch ? load_page_batch<SEFF, FP4>(kBatch, X0, X1, w, lane, pre, lens, p) : 0;

  // This warp's q rows of a unit: one bulk copy into its raw-q buffer, completing on qbar.
  int q_issued = 0, q_done = 0;  // q copies issued / waited for (one in flight at most)
  auto q_fetch = [&](const Unit& u) {
    q_issued++;
    if (lane == 0) {
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(qbar, G * kD * 2);
      bulk_copy_g2s(smem_addr(qraw),
                    p.q + (static_cast<size_t>(u.b) * p.num_kv_heads * G + u.h * G) * kD,
                    G * kD * 2, qbar, 0ull);
    }
    __syncwarp();
  };
  // The units of the CTA's range: the first (uf) and the last (ul) may be shared with
  // other CTAs; the units between them lie wholly inside the range.
  Unit uf, ul;
  if (has_tiles) {
    unit_of_tile(uf, X0, pre, lens, p);
    unit_of_tile(ul, X1 - 1, pre, lens, p);
  }
  int x = X0 + w;
  Unit cu;
  if (x < X1) unit_of_tile(cu, x, pre, lens, p);
  // uf and ul have one copy of their q rows each, prepared by all warps together; only
  // units between them are prepared by the warp that walks them.
  auto is_uf = [&](const Unit& u) { return u.b == uf.b && u.h == uf.h; };
  auto is_ul = [&](const Unit& u) { return u.b == ul.b && u.h == ul.h; };
  const bool two_edges = has_tiles && !is_uf(ul);

  // Fused append: if this warp holds the last tile of its first unit and that unit's q
  // comes from a CTA table (its own fragment table is then free as the patch buffer), the
  // unit's new K/V rows are loaded, rotated and quantised before the wait: pure arithmetic
  // into shared memory, under the previous kernel's tail.  That kernel may be the one that
  // writes these rows, so they are read again after the wait, and quantised again if they
  // are not the same.  Other units do all of it at their segment's start.
  bool pre_quantised = false;
  uint2 kraw0 = make_uint2(0u, 0u), vraw0 = make_uint2(0u, 0u);
  auto new_row = [&](const __half* rows) {
    return load_new_row(rows + (static_cast<size_t>(cu.b) * p.num_kv_heads + cu.h) * kD, lane);
  };
  if constexpr (FUSED) {
    if (x < X1 && (is_uf(cu) || is_ul(cu))) {
      const int seg_end0 = min(X1, cu.U + cu.n);
      const int xl0 = x + kWarps * ((seg_end0 - x + kWarps - 1) / kWarps - 1);
      if (xl0 == cu.U + cu.n - 1) {
        kraw0 = new_row(p.k_new);
        vraw0 = new_row(p.v_new);
        fused_quantise<FP4>(kraw0, vraw0, lane, reinterpret_cast<uint8_t*>(frag), p);
        pre_quantised = true;
      }
    }
  }

  griddep_wait();

  uint2 kraw1 = kraw0, vraw1 = vraw0;
  if constexpr (FUSED) {
    if (pre_quantised) {  // (the same in the whole warp)
      kraw1 = new_row(p.k_new);
      vraw1 = new_row(p.v_new);
    }
  }

  // q goes ahead of the tile copies, so that it is not queued behind them; then the first
  // kStages tiles.
  if (has_tiles && tid == 0) {
    mbar_arrive_expect_tx(qbar_cta, (two_edges ? 2 : 1) * G * kD * 2);
    bulk_copy_g2s(smem_addr(qraw_all + kWarps * G * kD * 2),
                  p.q + (static_cast<size_t>(uf.b) * p.num_kv_heads * G + uf.h * G) * kD,
                  G * kD * 2, qbar_cta, 0ull);
    if (two_edges)
      bulk_copy_g2s(smem_addr(qraw_all + (kWarps + 1) * G * kD * 2),
                    p.q + (static_cast<size_t>(ul.b) * p.num_kv_heads * G + ul.h * G) * kD,
                    G * kD * 2, qbar_cta, 0ull);
  }
  if (x < X1 && !is_uf(cu) && !is_ul(cu)) q_fetch(cu);
  while (pr.t < pr.nT && pr.t < kStages)
    producer_issue<SEFF, FP4>(pr, X0, X1, w, lane, ring_s, bar_s, pol, pre, lens, p);

  // An empty sequence has no tiles: its output rows are zeros (CTAs share the writes).
  const int row_words = p.num_kv_heads * G * kD / 8;  // 16-byte words per sequence
  for (int b = blockIdx.x; b < p.batch; b += p.total_ctas)
    if (pre[b + 1] == pre[b])
      for (int i = tid; i < row_words; i += kThreads)
        reinterpret_cast<uint4*>(p.out + static_cast<size_t>(b) * p.num_kv_heads * G * kD)[i] =
            make_uint4(0u, 0u, 0u, 0u);
  if (!has_tiles) return;  // the whole CTA (no copies were issued): nothing else to do

  // A warp's partial of uf goes to its part of the merge buffer and its partial of ul
  // (always its last segment, when its ring has drained) to its ring's first slot;
  // partials of the units between go to the warp's global slot.  All of them are merged
  // at the CTA's end.
  const int unit_f = uf.b * p.num_kv_heads + uf.h;
  const int unit_l = ul.b * p.num_kv_heads + ul.h;
  auto out_row = [&](int b, int h) {
    return p.out + (static_cast<size_t>(b) * p.num_kv_heads * G + h * G) * kD;
  };
  auto warp_slot = [&](int unit, int ww) {
    return p.part + (static_cast<size_t>(unit + kc) * kWarps + ww) * G * kPartStride;
  };
  float* const rec_f = mbuf;                             // [kWarps][G][kPartStride]
  float* const rec_l = reinterpret_cast<float*>(ring);   // warp ww's: + ww*kStages*kSlot

  int consumed = 0;   // tiles of this warp consumed (tile t uses slot t % kStages)
  bool dead = false;  // a bounded wait gave up: stop touching the ring
  // uf's and ul's q rows: every warp rotates and slices its share of the queries.
  if (!mbar_wait_warp(qbar_cta, 0u, kWaitLimitNs)) dead = true;
  if (!dead)
    for (int t = 0; t < (two_edges ? 2 : 1); t++)
      prep_q<G, kWarps, FP4>(qraw_all + (kWarps + t) * G * kD * 2, frag_all + (kWarps + t) * kFragWords,
                             sf_all + (kWarps + t) * 8, lane, p, w);
  if (dead && lane == 0) atomicOr(p.status, KVQ_DEV_TIMEOUT_BIT);
  __syncthreads();
  if constexpr (FUSED) {
    if (pre_quantised &&
        __any_sync(kFull, kraw0.x != kraw1.x || kraw0.y != kraw1.y || vraw0.x != vraw1.x || vraw0.y != vraw1.y))
      fused_quantise<FP4>(kraw1, vraw1, lane, reinterpret_cast<uint8_t*>(frag), p);
  }
  State<G> st;
  state_reset<G>(st);
  typename QF<G, FP4>::type qf;
  constexpr int NQ = QFrag<G>::NQ;
  while (x < X1) {
    const int seg_end = min(X1, cu.U + cu.n);
    const int nt = (seg_end - x + kWarps - 1) / kWarps;
    const int x_next = x + kWarps * nt;
    const bool has_next = x_next < X1;
    Unit nu = cu;
    if (has_next) unit_of_tile(nu, x_next, pre, lens, p);
    // q of this unit: rotate and slice into the warp's fragment table; then fetch the
    // next unit's rows into the freed buffer.
    const int table = is_uf(cu) ? kWarps : (is_ul(cu) ? kWarps + 1 : -1);
    if (table >= 0) {
      qfrag_get<G>(qf, frag_all + table * kFragWords, sf_all + table * 8, lane);
    } else {
      if (!dead) {
        if (mbar_wait_warp(qbar, static_cast<uint32_t>(q_done & 1), kWaitLimitNs)) q_done++;
        else dead = true;
      }
      if (!dead) prep_q<G, 1, FP4>(qraw, frag, sf, lane, p);
      qfrag_get<G>(qf, frag, sf, lane);
    }
    if (has_next && !dead && !is_ul(nu)) q_fetch(nu);
    state_reset<G>(st);
    // Fused append: the warp holding the unit's last tile rotates, quantises and stores the
    // unit's new token, and patches it into that tile's slot once the slot has landed.
    bool new_ok = false;
    if constexpr (FUSED) {
      const int xl = x + kWarps * (nt - 1);  // this warp's last tile of the unit
      uint8_t* patch = reinterpret_cast<uint8_t*>(frag);  // free until the next unit's q
      if (xl == cu.U + cu.n - 1 && !dead) {
        if (!(pre_quantised && x == X0 + w)) fused_quantise<FP4>(new_row(p.k_new), new_row(p.v_new), lane, patch, p);
        new_ok = fused_store<FP4>(cu.b, cu.h, lane, patch, p);
        if (lane == 0)
          *reinterpret_cast<int*>(patch + PatchLayout<FP4>::kJ) = cu.L - 1 - (xl - cu.U) * kTileTokens;
        __syncwarp();
      }
    }

    // (As a prefix of each half for INT4, of the tile for NVFP4: either form costs the other format
    // 2 to 6 % of its time in register moves.)
    auto ntok_of = [&](int xx) {
      const int n = min(kTileTokens, cu.L - (xx - cu.U) * kTileTokens);
      if constexpr (FP4) return n;
      else return Valid{{n, n - 16}};
    };
    // Release a consumed slot and refill it with the warp's tile kStages ahead.
    auto refill = [&]() {
      __syncwarp();
      if (pr.t < pr.nT) {
        fence_proxy_async_smem();
        producer_issue<SEFF, FP4>(pr, X0, X1, w, lane, ring_s, bar_s, pol, pre, lens, p);
      }
    };
    float sc[2][NQ][2];
    int slot_i = consumed % kStages;
    uint32_t parity = static_cast<uint32_t>((consumed / kStages) & 1);
    if (!dead) {
      if (!mbar_wait_warp(bar_s + 8 * slot_i, parity, kWaitLimitNs)) {
        dead = true;
      } else {
        if constexpr (FUSED) {
          if (new_ok && nt == 1)
            patch_slot<SEFF, FP4>(ring_w + slot_i * kSlot, lane, reinterpret_cast<const uint8_t*>(frag));
        }
        tile_qk_any<G, SEFF>(qf, ring_p + slot_i * kSlot, ntok_of(x), lane, sc);
        float alpha[NQ];
        if (tile_softmax_stats<G>(st, sc, alpha)) tile_rescale<G>(st, alpha);
      }
    }
    // Steady state: a next tile of the unit always exists.  The QK^T and softmax statistics
    // of the next tile are computed next to the PV of the current one; only the rescale
    // of o' has to follow that PV.
    for (int i = 0; i + 1 < nt && !dead; i++) {
      const int xi = x + kWarps * i;
      const int cur = slot_i;
      const int nslot = cur + 1 == kStages ? 0 : cur + 1;
      const uint32_t npar = cur + 1 == kStages ? parity ^ 1u : parity;
      if (!mbar_wait_warp(bar_s + 8 * nslot, npar, kWaitLimitNs)) {
        dead = true;
        break;
      }
      float sn[2][NQ][2], alpha[NQ];
      if constexpr (FUSED) {
        if (new_ok && i + 2 == nt)
          patch_slot<SEFF, FP4>(ring_w + nslot * kSlot, lane, reinterpret_cast<const uint8_t*>(frag));
      }
      tile_qk_any<G, SEFF>(qf, ring_p + nslot * kSlot, ntok_of(xi + kWarps), lane, sn);
      const bool rescale = tile_softmax_stats<G>(st, sn, alpha);
      tile_pv_any<G, SEFF, FP4>(st, ring_p + cur * kSlot, ntok_of(xi), lane, sc);
      consumed++;
      slot_i = nslot;
      parity = npar;
      refill();
      if (rescale) tile_rescale<G>(st, alpha);
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int qq = 0; qq < NQ; qq++)
#pragma unroll
          for (int r = 0; r < 2; r++) sc[j][qq][r] = sn[j][qq][r];
    }
    if (!dead) {  // last tile of the unit for this warp
      tile_pv_any<G, SEFF, FP4>(st, ring_p + slot_i * kSlot, ntok_of(x + kWarps * (nt - 1)), lane, sc);
      consumed++;
      refill();
    }
    if (dead && lane == 0) atomicOr(p.status, KVQ_DEV_TIMEOUT_BIT);

    const int unit = cu.b * p.num_kv_heads + cu.h;
    if (cu.n == 1) {
      // This warp is the unit's only contributor: finish it now (the fragment table is
      // free until the next unit's q is prepared).
      finish_from_state<G>(st, reinterpret_cast<float*>(frag), out_row(cu.b, cu.h), lane, p);
    } else if (unit == unit_f) {
      state_write<G>(st, rec_f + w * G * kPartStride, lane);
    } else if (unit == unit_l) {
      state_write<G>(st, rec_l + w * (kStages * kSlot / 4), lane);
    } else {
      state_write<G>(st, warp_slot(unit, w), lane);
    }
    x = x_next;
    cu = nu;
  }

  // ---- CTA end: every partial of the range is written (shared or global memory).
  __syncthreads();
  // The (one or two) edge units: merge the warps' partials from shared memory, queries
  // split over the warps.  A unit inside the range is finished here; a shared one leaves
  // one record per CTA at the CTA's slot (warp slot 0).
  const int nedge = unit_l == unit_f ? 1 : 2;
  bool shared_edge[2] = {false, false};
#pragma unroll
  for (int e = 0; e < 2; e++) {
    if (e >= nedge) break;
    const Unit& u = e == 0 ? uf : ul;
    const int unit = e == 0 ? unit_f : unit_l;
    const int a = max(X0, u.U), c = min(X1, u.U + u.n) - a;  // this CTA's tiles of u
    shared_edge[e] = !(u.U >= X0 && u.U + u.n <= X1);
    if (u.n == 1) continue;  // already finished by its warp
    float* base = e == 0 ? rec_f : rec_l;
    const int wstride = e == 0 ? G * kPartStride : kStages * kSlot / 4;
    auto rec = [&](int j) -> const float* { return base + ((a - X0 + j) & (kWarps - 1)) * wstride; };
    merge_few<G, kWarps, false, kWarps>(min(kWarps, c), rec, w, out_row(u.b, u.h),
                                        shared_edge[e] ? warp_slot(unit, 0) : nullptr, lane, p);
  }
  // Units between the edges (wholly inside the range, at least two tiles): their warps'
  // records are in global memory; warp w merges every kWarps-th of them.
  if (nedge == 2) {
    Unit u = uf;
    unit_next(u, pre, lens, p);
    for (int i = 0; !(u.b == ul.b && u.h == ul.h); i++, unit_next(u, pre, lens, p)) {
      if ((i & (kWarps - 1)) != w || u.n == 1) continue;
      const int unit = u.b * p.num_kv_heads + u.h;
      auto rec = [&](int j) -> const float* { return warp_slot(unit, (u.U - X0 + j) & (kWarps - 1)); };
      merge_few<G, 1, true, kWarps>(min(kWarps, u.n), rec, 0, out_row(u.b, u.h), nullptr, lane, p);
    }
  }
  // Shared edge units: publish this CTA's record (a CTA barrier, then one acquire-release
  // arrival per unit); the last of the unit's CTAs merges.
  if (shared_edge[0] || shared_edge[1]) {
    __syncthreads();
    if (lane == 0 && w < nedge && shared_edge[w]) {
      const Unit& u = w == 0 ? uf : ul;
      const int unit = w == 0 ? unit_f : unit_l;
      const int ncta = (u.U + u.n - 1) / chunk - u.U / chunk + 1;
      const int old = atom_add_acq_rel_gpu(p.counters + unit, 1);
      const int last = old == ncta - 1;
      if (last) p.counters[unit] = 0;  // ready for the next call
      last_flag_e[w] = last;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; e++) {
      if (e >= nedge || !shared_edge[e] || !last_flag_e[e]) continue;
      const Unit& u = e == 0 ? uf : ul;
      const int unit = e == 0 ? unit_f : unit_l;
      const int k0 = u.U / chunk, ncta = (u.U + u.n - 1) / chunk - k0 + 1;
      auto rec = [&](int j) -> const float* {
        return p.part + (static_cast<size_t>(unit + k0 + j) * kWarps) * G * kPartStride;
      };
      if (ncta <= 8)
        merge_few<G, kWarps, true, 8>(ncta, rec, w, out_row(u.b, u.h), nullptr, lane, p);
      else
        merge_records<G, kWarps, true>(ncta, rec, w, out_row(u.b, u.h), nullptr, lane, p);
    }
  }

  if (dead) {
    // Let copies still in flight land before the CTA's shared memory is released.
    for (int j = consumed; j < pr.t; j++)
      mbar_wait_warp(bar_s + 8 * (j % kStages), static_cast<uint32_t>((j / kStages) & 1),
                        kWaitLimitNs);
    for (; q_done < q_issued; q_done++)
      mbar_wait_warp(qbar, static_cast<uint32_t>(q_done & 1), kWaitLimitNs);
    mbar_wait_warp(qbar_cta, 0u, kWaitLimitNs);
  }
}

template <int G, int SEFF>
void* kernel_ptr(bool fused, bool fp4) {
  if (fp4)
    return fused ? reinterpret_cast<void*>(&decode_kernel<G, SEFF, true, true>)
                 : reinterpret_cast<void*>(&decode_kernel<G, SEFF, false, true>);
  return fused ? reinterpret_cast<void*>(&decode_kernel<G, SEFF, true, false>)
               : reinterpret_cast<void*>(&decode_kernel<G, SEFF, false, false>);
}

void* pick_kernel(int group, int seff, bool fused, bool fp4) {
#define KVQ_PICK(GG)                                         \
  if (group == GG) {                                         \
    if (seff == 16) return kernel_ptr<GG, 16>(fused, fp4);   \
    if (seff == 32) return kernel_ptr<GG, 32>(fused, fp4);   \
  }
  KVQ_PICK(1)
  KVQ_PICK(2)
  KVQ_PICK(4)
  KVQ_PICK(8)
#undef KVQ_PICK
  return nullptr;
}

size_t smem_bytes(int group, int max_batch, bool fp4) {
  size_t s = static_cast<size_t>(kWarps) * kStages * slot_bytes(fp4);  // rings
  s += static_cast<size_t>(kWarps + 2) * group * kD * 2;             // raw q rows
  s += sizeof(uint32_t) * (kWarps + 2) * frag_words(group, fp4);     // q fragment tables
  s += sizeof(float) * (kWarps + 2) * 8;                             // M factors
  s += sizeof(float) * kWarps * group * kPartStride;                 // CTA merge buffer
  s += sizeof(uint64_t) * (kWarps * (kStages + 1) + 1);              // mbarriers
  s += static_cast<size_t>(2 * max_batch + 1) * sizeof(int32_t);     // prefix, lengths
  s += 128;                                                          // alignment slack
  return (s + 15) & ~static_cast<size_t>(15);
}

}  // namespace

int plan_decode(int group, int page_size, int max_batch, int num_sms, int fp4, DecodeLaunch* out) {
  const int seff = page_size < kTileTokens ? page_size : kTileTokens;
  const size_t smem = smem_bytes(group, max_batch, fp4 != 0);
  // The dynamic shared memory cap of the variants is set to the most any call of this
  // library uses (max_batch 4096), so plans made for several caches never shrink it
  // under one another; the grid is the smaller occupancy of the variants (plain and
  // fused).
  const size_t cap_bytes = smem_bytes(group, 4096, fp4 != 0);
  int occ = 3;
  for (int fused = 0; fused < 2; fused++) {
    void* fn = pick_kernel(group, seff, fused != 0, fp4 != 0);
    if (!fn) return -1;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(cap_bytes)) != cudaSuccess)
      return -2;
    int o = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, fn, kThreads, smem) != cudaSuccess)
      return -2;
    if (o < occ) occ = o;
  }
  if (occ < 1) return -1;
  out->grid = num_sms * occ;
  out->smem = smem;
  return 0;
}

int launch_decode(const DecodeParams& p, const DecodeLaunch& L, cudaStream_t stream) {
  const int seff = p.page_size < kTileTokens ? p.page_size : kTileTokens;
  void* fn = pick_kernel(p.group, seff, p.k_new != nullptr, p.fp4 != 0);
  if (!fn) return -1;
  DecodeParams q = p;
  q.total_ctas = L.grid;
  void* args[] = {&q};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(L.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) return -2;
  return 0;
}

}  // namespace kvq
