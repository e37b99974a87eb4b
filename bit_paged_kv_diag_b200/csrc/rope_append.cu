// rope_append.cu -- append of K and V to the paged 4-bit cache with the position rotation of
// q and k applied on the way, for sm_100a.
//
// Mathematics.  Token at position p, pair i of the rotary_dim / 2 rotated channel pairs:
// theta = p * inv_freq[i] in fp64, c = fl32(factor cos theta), s = fl32(factor sin theta), and
//   x'_a = x_a c - x_b s,  x'_b = x_b c + x_a s
// with (a, b) = (i, i + rotary_dim / 2), or (2i, 2i + 1) for the interleaved form.  The angle
// is formed in fp64 because an fp32 product of a far position loses the angle itself (2^17
// tokens times 1 leaves 2^-7 radian).  For k both products and the sum round to fp32 one by one,
// so that the stored codes are those of any implementation that rounds the same way from the same
// cosines and sines (these may round apart by a step of fp32, which moves at most one code in 10^5 by
// one); k' stays in fp32 on its way into the block-diagonal Hadamard butterfly and the quantiser (append_row.cuh),
// which are the append kernel's.  For q the sum is one fma; q' is rounded once to fp16, the type
// that the attention calls read.
//
// Layout.  A CTA takes a few tokens (of all heads, or of some when the call is short): their K
// and V rows come by bulk copies into shared memory, the angles of the tokens are computed once
// for all heads into a table there, and its warps take stages of 16 rows.
//   q: 8 lanes a row, lane j the two 8-channel chunks of the pairs 8 j .. 8 j + 7, so a pair
//      never leaves a lane and the cosines stay in registers from row to row; global memory to
//      registers and back, no shared memory (a row costs 22 warp instructions; two lanes a row,
//      each computing both partners' products, cost 77).
//   k, v: two lanes a row, as in the append kernel.  (Eight lanes a row straight from global memory
//      repeat the scale's divisions and the addresses four times as often: 349 us against 303.)
// Measured, the kernel alone behind a flush of L2, 8 x 8192 tokens, 32 + 2 x 8 heads, INT4, b = 128:
// 262 us, 5.4 TB/s of algorithmic
// bytes, 0.82 of the copy rate; 132 M warp instructions at 46 % of the issue slots with 16 warps per
// SM.  One token for each of 16 sequences: 7.9 us, of which about 2 us are the chain of offsets,
// length and page, and much of the rest instruction fetches: the form of the pairs is a template
// parameter because the smaller code took 9.0 us down to 7.9 (and 274 to 262).  Not kept: one
// persistent CTA per slot with the next tile's copies in flight (registers spill: 503 us); copies
// issued only after the tokens' places are known (352 us); q rows loaded a stage ahead (266 us).
// (NVFP4 with b = 128 spills 4 to 8 bytes at the 128 registers of four CTAs per SM.)
#include <cuda_fp16.h>
#include <stdint.h>

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
constexpr int kTileRows = 128;        // K and V rows of a CTA's tile, about 32 KB
constexpr int kRopeTokens = 32;       // tokens of a tile at most: a lane each
constexpr int kMaxSmem = (kTileRows + 2 * 15) * kRow + kRopeTokens * (kD * 4 + 16) + 16;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // bounded waits: 2 s

constexpr int kSlotBadPos = -1, kSlotPadding = -2;

// Per token of the tile: where its rows go, and its angle's position.
struct TokenDest {
  int page;  // pool page, or -1
  int slot;  // slot of the page, or kSlotBadPos / kSlotPadding
  int pos;   // position of the angle
  int pad;   // (16 bytes)
};

__host__ __device__ inline int round16(int n) { return (n + 15) & ~15; }

// Rows of one kind, padded to whole warp stages.
__host__ __device__ inline size_t tile_smem(int tokens, int heads) {
  return static_cast<size_t>(2 * round16(tokens * heads)) * kRow +
         static_cast<size_t>(tokens) * (2 * (kD / 2) * 4 + sizeof(TokenDest)) + 16;
}

// cos and sin of theta >= 0 or < 0, |theta| < 2^31, to about 2^-48: theta less the nearest multiple
// n of pi / 2 (whose first 53 bits and next 53 are subtracted by one fma each, so that r keeps an
// absolute error of 2^-53), then Taylor's series on |r| <= pi / 4 (first terms left out: r^17 / 17!
// and r^18 / 18!, below 2^-53), swapped and signed by n mod 4.
__device__ __forceinline__ void cos_sin(double theta, double& c, double& s) {
  const double n = rint(theta * 0.63661977236758134308);
  double r = fma(-n, 1.5707963267948965580, theta);
  r = fma(-n, 6.1232339957367658861e-17, r);
  const double z = r * r;
  double cp = 1.0 / 20922789888000.0, sp = -1.0 / 1307674368000.0;
  cp = fma(cp, z, -1.0 / 87178291200.0);
  sp = fma(sp, z, 1.0 / 6227020800.0);
  cp = fma(cp, z, 1.0 / 479001600.0);
  sp = fma(sp, z, -1.0 / 39916800.0);
  cp = fma(cp, z, -1.0 / 3628800.0);
  sp = fma(sp, z, 1.0 / 362880.0);
  cp = fma(cp, z, 1.0 / 40320.0);
  sp = fma(sp, z, -1.0 / 5040.0);
  cp = fma(cp, z, -1.0 / 720.0);
  sp = fma(sp, z, 1.0 / 120.0);
  cp = fma(cp, z, 1.0 / 24.0);
  sp = fma(sp, z, -1.0 / 6.0);
  cp = fma(cp, z, -0.5);
  cp = fma(cp, z, 1.0);
  sp = fma(sp * z, r, r);
  const int m = static_cast<int>(static_cast<long long>(n));
  c = (m & 1) ? sp : cp;
  s = (m & 1) ? cp : sp;
  if ((m + 1) & 2) c = -c;
  if (m & 2) s = -s;
}

// Two 16-bit values of a word -> fp32 pair, exact.
template <bool BF16>
__device__ __forceinline__ f2 widen(uint32_t w) {
  if constexpr (BF16) return pk(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  else {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pk(v.x, v.y);
  }
}

// Position rotation of one lane's half row.  row: the row in shared memory; raw[t] = its chunk
// t ^ rho (of the lane's half l); cs: the token's cosines [64], then sines [64]; x[4t + e] =
// channels 2e, 2e + 1 of chunk t ^ rho after the rotation.  Chunks are 8 channels and
// rotary_dim is a multiple of 16, so a chunk's partner is a whole chunk.
template <bool BF16, bool INTER>
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
    if constexpr (!INTER) {
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

// Stage h = 1 of the butterfly: (a, c) -> (a + c, a - c) inside every pair.
template <int BLOCK>
__device__ __forceinline__ void first_stage(f2 (&x)[32]) {
  if constexpr (BLOCK > 1) {
#pragma unroll
    for (int i = 0; i < 32; i++) {
      float a, c;
      upk(x[i], a, c);
      x[i] = pk(__fadd_rn(a, c), __fsub_rn(a, c));
    }
  }
}

// 16 bytes of global memory that are read once.
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Two fp32 values -> fp16, nearest even (lo -> low half): one conversion of the pair (two scalar
// ones go through the special-function unit, which then bounds the q part).
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8 values of the inputs' type -> fp16.
template <bool BF16>
__device__ __forceinline__ uint4 half_chunk(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; e++) {
    float a, b;
    upk(widen<BF16>(w[e]), a, b);
    o[e] = half_pair(a, b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The rotation of two chunks a, b of 8 channels (16-bit values) with the 8 cosines and sines of
// their pairs: channel e of a with channel e of b, or, interleaved, the pairs inside the chunks.
template <bool BF16, bool INTER>
__device__ __forceinline__ void rotate_chunks(uint4& a, uint4& b, const f2 (&c)[4], const f2 (&s)[4]) {
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
  uint32_t oa[4], ob[4];
  if constexpr (!INTER) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const f2 x = widen<BF16>(wa[e]), y = widen<BF16>(wb[e]), ns = s[e] ^ 0x8000000080000000ull;
      float u0, u1, v0, v1;
      upk(fma2(y, ns, mul2(x, c[e])), u0, u1);
      upk(fma2(x, s[e], mul2(y, c[e])), v0, v1);
      oa[e] = half_pair(u0, u1);
      ob[e] = half_pair(v0, v1);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++) {
      float c0, c1, s0, s1;
      upk(c[e], c0, c1);
      upk(s[e], s0, s1);
#pragma unroll
      for (int i = 0; i < 2; i++) {  // pairs 2e, 2e + 1: chunk a for e < 2, chunk b after
        const int z = (2 * e + i) & 3;
        float x, y;
        upk(widen<BF16>(e < 2 ? wa[z] : wb[z]), x, y);
        const float cc = i ? c1 : c0, ss = i ? s1 : s0;
        (e < 2 ? oa : ob)[z] = half_pair(__fmaf_rn(y, -ss, __fmul_rn(x, cc)), __fmaf_rn(x, ss, __fmul_rn(y, cc)));
      }
    }
  }
  a = make_uint4(oa[0], oa[1], oa[2], oa[3]);
  b = make_uint4(ob[0], ob[1], ob[2], ob[3]);
}

template <int BLOCK, bool FP4, bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) rope_append_kernel(RopeAppendParams p) {
  griddep_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int t0 = blockIdx.x * p.tile_tokens, nt = min(p.tile_tokens, p.total_new_tokens - t0);
  const int h0 = blockIdx.y * p.tile_heads, nh = min(p.tile_heads, p.num_kv_heads - h0);
  const int gq = p.q ? nh * p.group : 0;  // q rows per token of this CTA
  const int nk = nt * nh, nq = nt * gq;
  // [K rows][V rows], each padded to 16 rows | cosines and sines | destinations | barrier
  const uint32_t k_s = smem_addr(smem), v_s = k_s + round16(nk) * kRow;
  uint8_t* const tail = smem + 2 * round16(nk) * kRow;
  float* const cs = reinterpret_cast<float*>(tail);
  TokenDest* const dest = reinterpret_cast<TokenDest*>(cs + nt * kD);
  const uint32_t bar = smem_addr(dest + nt);
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  griddep_wait();
  if (tid == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(2 * nk) * kRow);
  __syncthreads();
  // One bulk copy per token and kind: a token's heads are contiguous.
  for (int i = tid; i < 2 * nt; i += kThreads) {
    const int kind = i >= nt, t = kind ? i - nt : i;
    const uint8_t* src = static_cast<const uint8_t*>(kind ? p.v : p.k);
    src += static_cast<int64_t>(t0 + t) * (kind ? p.v_stride : p.k_stride) * 2 + static_cast<int64_t>(h0) * kRow;
    bulk_copy_g2s((kind ? v_s : k_s) + t * nh * kRow, src, nh * kRow, bar, l2_policy_evict_first());
  }
  // Each token's sequence, destination and position: a lane per token.
  if (w == 0) {
    const int t = t0 + lane;
    int first, next;
    const SeqWindow win = seq_window(p.cu_new_tokens, p.batch, t0);
    const int b = seq_find(win, p.cu_new_tokens, p.batch, t, first, next);
    if (lane < nt) {
      TokenDest d = {-1, kSlotPadding, 0, 0};
      if (t >= first && t < next) {
        const long long pos = static_cast<long long>(__ldg(p.seq_lens + b)) + (t - first);
        d.pos = p.positions ? __ldg(p.positions + t) : static_cast<int>(pos);
        d.slot = kSlotBadPos;
        if (pos >= 0 && (pos >> p.page_shift) < p.max_pages_per_seq) {
          d.slot = static_cast<int>(pos) & (p.page_size - 1);
          d.page = __ldg(p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq + (pos >> p.page_shift));
        }
        if (d.slot < 0) atomicOr(p.status, KVQ_DEV_BAD_POS_BIT);
        else if (d.page < 0 || d.page >= p.num_pages) {
          atomicOr(p.status, KVQ_DEV_BAD_PAGE_BIT);
          d.page = -1;
        }
      }
      dest[lane] = d;
    }
  }
  __syncthreads();
  const int pairs = p.rotary_dim >> 1;
  for (int i = tid; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, f = i - t * pairs;
    double s, c;
    cos_sin(static_cast<double>(dest[t].pos) * static_cast<double>(__ldg(p.inv_freq + f)), c, s);
    cs[t * kD + f] = static_cast<float>(c * p.factor);
    cs[t * kD + kD / 2 + f] = static_cast<float>(s * p.factor);
  }
  __syncthreads();

  // q: rows r of the tile, token r / gq.  Lane group lane / 8 takes four neighbouring rows of a
  // stage, all loaded before the first is rotated.
  const int nsq = (nq + kStageRows - 1) / kStageRows;
  {
    const int j = lane & 7, tasks = p.rotary_dim >> 4;
    const bool turn = j < tasks;
    const int ca = turn && !INTER ? j : 2 * j, cb = turn && !INTER ? j + tasks : 2 * j + 1;
    const uint8_t* const q0 = static_cast<const uint8_t*>(p.q) + static_cast<int64_t>(t0) * p.q_stride * 2 +
                              static_cast<int64_t>(h0) * p.group * kRow;
    uint8_t* const o0 = reinterpret_cast<uint8_t*>(p.q_out) +
                        (static_cast<size_t>(t0) * p.num_kv_heads + h0) * p.group * kRow;
    const size_t o_stride = static_cast<size_t>(p.num_kv_heads) * p.group * kRow;
    // The angles of token ti for this lane's pairs.
    auto angles = [&](int ti, f2 (&c)[4], f2 (&s)[4]) {
      const ulonglong2* src = reinterpret_cast<const ulonglong2*>(cs + ti * kD + 8 * j);
      const ulonglong2 c0 = src[0], c1 = src[1], s0 = src[kD / 8], s1 = src[kD / 8 + 1];
      c[0] = c0.x, c[1] = c0.y, c[2] = c1.x, c[3] = c1.y;
      s[0] = s0.x, s[1] = s0.y, s[2] = s1.x, s[3] = s1.y;
    };
    // One row's chunks, rotated (or only converted: channels behind rotary_dim), stored to dst.
    auto finish = [&](uint4& a, uint4& b, const f2 (&c)[4], const f2 (&s)[4], uint8_t* dst) {
      if (turn) {
        rotate_chunks<BF16, INTER>(a, b, c, s);
      } else if (BF16) {
        a = half_chunk<BF16>(a);
        b = half_chunk<BF16>(b);
      }
      stg_128(dst + 16 * ca, a.x, a.y, a.z, a.w);
      stg_128(dst + 16 * cb, b.x, b.y, b.z, b.w);
    };
    if ((gq & 3) == 0) {  // a lane's four rows belong to one token: one address, one read of its angles
      for (int st = w; st < nsq; st += kWarps) {
        const int r0 = st * kStageRows + 4 * (lane >> 3), ti = r0 / gq;
        if (r0 >= nq) continue;
        const uint8_t* const src = q0 + static_cast<int64_t>(ti) * p.q_stride * 2 + (r0 - ti * gq) * kRow;
        uint8_t* const dst = o0 + ti * o_stride + (r0 - ti * gq) * kRow;
        uint4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          a[i] = ldg_stream(src + i * kRow + 16 * ca);
          b[i] = ldg_stream(src + i * kRow + 16 * cb);
        }
        f2 c[4], s[4];
        angles(ti, c, s);
        if (dest[ti].slot == kSlotPadding) continue;
#pragma unroll
        for (int i = 0; i < 4; i++) finish(a[i], b[i], c, s, dst + i * kRow);
      }
    } else {  // (few heads: a row at a time)
#pragma unroll 1
      for (int r = 4 * w + (lane >> 3); r < nq; r += 4 * kWarps) {
        const int ti = r / gq;
        const uint8_t* const src = q0 + static_cast<int64_t>(ti) * p.q_stride * 2 + (r - ti * gq) * kRow;
        uint4 a = ldg_stream(src + 16 * ca), b = ldg_stream(src + 16 * cb);
        f2 c[4], s[4];
        angles(ti, c, s);
        if (dest[ti].slot != kSlotPadding) finish(a, b, c, s, o0 + ti * o_stride + (r - ti * gq) * kRow);
      }
    }
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
  const int nsk = round16(nk) / kStageRows;
  const uint32_t cs_s = smem_addr(cs);
  // (the warps that had a q stage less start here)
  for (int st = (w + nsq) % kWarps; st < 2 * nsk; st += kWarps) {
    const int kind = st >= nsk;
    const int r = (kind ? st - nsk : st) * kStageRows + (lane >> 1);
    const uint32_t row = (kind ? v_s : k_s) + r * kRow;
    const bool active = r < nk;
    uint4 raw[8];
    f2 x[32];
    int ti = 0;
    if (active) {  // both lanes of a row take the same branch
      ti = r / nh;
#pragma unroll
      for (int t = 0; t < 8; t++) raw[t] = lds_128(row + kD * l + 16 * (t ^ rho));
    }
    if (active) {
      if (kind == 0) {
        rope_row<BF16, INTER>(raw, row, cs_s + ti * (kD * 4), rho, l, p, x);
        first_stage<BLOCK>(x);
        rotate_stages<BLOCK>(rho, l, pmask, x);
      } else if constexpr (BF16) {
#pragma unroll
        for (int t = 0; t < 8; t++) {
          const uint32_t wd[4] = {raw[t].x, raw[t].y, raw[t].z, raw[t].w};
#pragma unroll
          for (int e = 0; e < 4; e++) x[4 * t + e] = widen<BF16>(wd[e]);
        }
        first_stage<BLOCK>(x);
        rotate_stages<BLOCK>(rho, l, pmask, x);
      } else {
        rotate_row<BLOCK>(raw, rho, l, pmask, x);
      }
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

template <int BLOCK, bool FP4, bool BF16, bool INTER>
int launch_one(const cudaLaunchConfig_t& cfg, const RopeAppendParams& p) {
  if (!ensure_smem<rope_append_kernel<BLOCK, FP4, BF16, INTER>>(kMaxSmem)) return -2;
  return cudaLaunchKernelEx(&cfg, rope_append_kernel<BLOCK, FP4, BF16, INTER>, p) == cudaSuccess ? 0 : -2;
}

template <int BLOCK, bool FP4>
int launch_type(const cudaLaunchConfig_t& cfg, const RopeAppendParams& p, bool bf16) {
  if (p.interleaved)
    return bf16 ? launch_one<BLOCK, FP4, true, true>(cfg, p) : launch_one<BLOCK, FP4, false, true>(cfg, p);
  return bf16 ? launch_one<BLOCK, FP4, true, false>(cfg, p) : launch_one<BLOCK, FP4, false, false>(cfg, p);
}

template <bool FP4>
int launch_block(const cudaLaunchConfig_t& cfg, const RopeAppendParams& p, int block, bool bf16) {
  switch (block) {
    case 1: return launch_type<1, FP4>(cfg, p, bf16);
    case 32: return launch_type<32, FP4>(cfg, p, bf16);
    case 64: return launch_type<64, FP4>(cfg, p, bf16);
    case 128: return launch_type<128, FP4>(cfg, p, bf16);
    default: return -1;
  }
}

}  // namespace

int launch_rope_append(RopeAppendParams p, int block, bool fp4, bool bf16, int num_sms, cudaStream_t stream) {
  if (p.total_new_tokens == 0) return 0;
  int heads = kTileRows / 2;
  if (heads > p.num_kv_heads) heads = p.num_kv_heads;
  int tokens = kTileRows / (2 * heads);
  if (tokens > kRopeTokens) tokens = kRopeTokens;
  // A short call is spread over the SMs' four CTAs each, in one wave: tiles of fewer tokens, then of
  // fewer heads.  (2,580 tokens, 40 heads: 8 tokens a tile 19.8 us, 5 a tile 19.1 us.)
  const int slots = 4 * num_sms, spread = (p.total_new_tokens + slots - 1) / slots;
  if (tokens > spread) tokens = spread;
  auto ctas = [&] {
    return static_cast<long long>((p.total_new_tokens + tokens - 1) / tokens) * ((p.num_kv_heads + heads - 1) / heads);
  };
  while (heads > 1 && ctas() < num_sms) heads = (heads + 1) / 2;
  p.tile_tokens = tokens;
  p.tile_heads = heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.total_new_tokens + tokens - 1) / tokens, (p.num_kv_heads + heads - 1) / heads);
  if (cfg.gridDim.y > 65535) return -1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = tile_smem(tokens, heads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return fp4 ? launch_block<true>(cfg, p, block, bf16) : launch_block<false>(cfg, p, block, bf16);
}

}  // namespace kvq
