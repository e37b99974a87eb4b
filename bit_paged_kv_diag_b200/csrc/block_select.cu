// block_select.cu -- the pages that each query and KV head attends, chosen by an upper bound of
// q.k over the page's keys, q rounded to int8, for sm_100a.
//
// Mathematics.  Every query head's q is rotated with the cache's transform (y = c_b * butterfly,
// fp32, fixed order) and cut to int8: s = fl(max_d |y_d| / 127), c_d = rint(fl(y_d / s)), 0 when
// s = 0.  With a page's bounds lo_d, hi_d (int8) and sigma (a power of two),
//   I_g = sum_d max(c_d, 0) hi_d + min(c_d, 0) lo_d,   score = max_g fl(I_g s_g) * sigma
// over the query heads g of the KV head: for each g, sum_d c_d k_d <= I_g sigma for every key of
// the page.  |I_g| <= 127 * 127 * 128 < 2^24, so the integer sum is exact in any order and in
// fp32, and the choice does not depend on the split of the work.  Of the n pages at or before the
// query's position the first `sink` and the last `recent` are always taken, and the rest by
// score, a tie going to the lower page; with n <= num_blocks all pages are taken.
//
// Scores.  I is a product of the rows of all query heads of a tile (256 int8: min(c, 0), then
// max(c, 0)) with the pages' (256 int8: lo, then hi): mma.sync m16n8k32 s8.  Pages are the N side:
// a fragment is then one register pair of a page's row, and a 32-byte load from global memory is
// four fragments as it lands (as the M side its registers had to be regrouped for every product,
// three moves per MMA).  The query rows lie in shared memory in fragment order, one 16-byte load
// per 4 MMAs.  A dot product does not depend on the order of its terms, so lane c of a quad takes
// bytes 128 i + 32 c on: a load touches 8 whole 128-byte lines (16-byte loads took three times
// the passes through the L1 data path, which bounds this phase).  The heads of a query sit in
// rows R and R + 8, so that half of the maximum over the group stays inside a lane.
//
// Choice.  Keys are the scores as ordered 32-bit integers.  The k-th largest is found by counting
// the keys in 256 equal bins between the smallest and the largest, then inside the bin where the
// k-th falls, and so on: the range shrinks by 2^8 a round, and the search ends as soon as a bin is
// taken whole, or its keys fit a warp and are ranked against one another (a bisection takes about
// 20 passes over the keys).  The
// pages are then written in ascending order from ballot masks.  A team of warps shares a query.
//
// Measured, the kernel alone behind a flush of L2: 464 queries, 8 KV heads, G = 4, up to 1024 pages, on
// a page table of that width: 37 us in one wave of 264 CTAs, about
// a third each for q's codes, the scores and the choice, all of it dependency chains (16 warps per
// SM at 128 registers, 43 % of the issue slots; the integer MMAs are busy for 20 %).
// One decode step of 4 sequences of up to 2048 pages, 4 KV heads, G = 8: 12 us, of which the launch
// and the memory round trips to the first page rows are half.
// The tile and the cluster are planned from the width of the page table, all that the host knows: a
// wider table leaves fewer queries a tile.  The same chunk on tables of 2048, 4096 and 8192 pages: 1.06,
// 1.5 and 2.7 times the time; the decode step on 8192: 1.01 times.
//
// Few queries: a cluster of up to 8 CTAs shares the pages of one tile, and its first CTA collects
// the keys through distributed shared memory and makes the choice.
#include <cuda_fp16.h>
#include <stdint.h>

#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

namespace {

constexpr int kD = 128;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxQueries = 16;                // queries of a tile
constexpr int kBins = 256;
constexpr float kMagic = 12582912.0f;           // 1.5 * 2^23; |I| <= 127 * 127 * 128 < 2^21
constexpr int kMagicBits = 0x4B400000;
constexpr int kRowBytes = 2 * kD;              // bytes of a query head's codes
constexpr int kMaxCluster = 8;
constexpr int kTilePages = 32;                 // pages of a warp's step: 4 MMA tiles of 8
constexpr unsigned kFull = 0xffffffffu;

__host__ __device__ inline int key_words(int pages) { return (pages + 127) / 128 * 128; }
// Words from one query's keys to the next: 8 queries' stores of the same pages hit different banks.
__host__ __device__ inline int key_stride(int pages) { return key_words(pages) + 8; }

// Query heads of a tile, in whole MMA tiles of 16 rows.
__host__ __device__ inline int tile_rows(int queries, int group) { return (queries * group + 15) / 16 * 16; }

inline size_t select_smem(int queries, int group, int pages) {
  return static_cast<size_t>(queries) * key_stride(pages) * 4 + tile_rows(queries, group) * (kRowBytes + 4);
}

constexpr size_t kSmemCap = 200 * 1024;

// Float -> integer of the same order; never 0, which marks the pages that are not a choice.
// (of fl(x s), s a power of two)
__device__ __forceinline__ uint32_t ordered(float x, float s) {
  const int b = __float_as_int(__fmaf_rn(x, s, 0.0f));  // -0 -> +0
  return max(static_cast<uint32_t>(b ^ ((b >> 31) | static_cast<int>(0x80000000u))), 1u);
}

// 32 bytes of global memory, as one load.  (Not a read-only load: with programmatic launches the
// kernel that writes these bytes may run after this one has started.)
__device__ __forceinline__ u32x8 ldg_256(const void* p) {
  u32x8 r;
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                 "=r"(r.w[7])
               : "l"(p));
  return r;
}

// Add 1 to a word of shared memory if `on` (predicated: no branch).
__device__ __forceinline__ void count_if(uint32_t addr, bool on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(addr),
               "r"(static_cast<uint32_t>(on))
               : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of a shared-memory location in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Bytes 4 x .. 4 x + 3 of row R of an MMA tile, in fragment order: byte 128 i + 32 c + 8 h + 4 u
// of a row belongs to k-step 4 i + h, lane 4 (R mod 8) + c, register 2 u + R / 8.
__device__ __forceinline__ void put_codes(uint32_t* tile, int R, int x, uint32_t v) {
  const int i = x >> 5, c = (x >> 3) & 3, h = (x >> 1) & 3, u = x & 1;
  tile[((4 * i + h) * 32 + 4 * (R & 7) + c) * 4 + 2 * u + (R >> 3)] = v;
}

// Codes and factors of kBatch query heads at once (their shuffle chains interleave), by one warp;
// raw[z]: channels 4 lane .. 4 lane + 3 of the head in row i0 + kWarps z of the MMA tiles.
template <int kBatch>
__device__ __forceinline__ void prep_rows(const uint2 (&raw)[kBatch], uint32_t* frag, float* sq, int i0, int nrow,
                                          int lane, const SelectParams& p) {
  float x[kBatch][4];
#pragma unroll
  for (int z = 0; z < kBatch; z++) {
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&raw[z].x));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&raw[z].y));
    const float a0 = __fadd_rn(lo.x, lo.y), a1 = __fsub_rn(lo.x, lo.y);
    const float a2 = __fadd_rn(hi.x, hi.y), a3 = __fsub_rn(hi.x, hi.y);
    const bool rot = p.hadamard_block > 1;
    x[z][0] = rot ? __fadd_rn(a0, a2) : lo.x;
    x[z][2] = rot ? __fsub_rn(a0, a2) : hi.x;
    x[z][1] = rot ? __fadd_rn(a1, a3) : lo.y;
    x[z][3] = rot ? __fsub_rn(a1, a3) : hi.y;
  }
#pragma unroll
  for (int s = 0; s < 5; s++) {
    if ((4 << s) < p.hadamard_block) {
      const float sgn = ((lane >> s) & 1) ? -1.0f : 1.0f;
#pragma unroll
      for (int z = 0; z < kBatch; z++)
#pragma unroll
        for (int e = 0; e < 4; e++) x[z][e] = __fmaf_rn(x[z][e], sgn, __shfl_xor_sync(kFull, x[z][e], 1 << s));
    }
  }
  float s[kBatch];
#pragma unroll
  for (int z = 0; z < kBatch; z++) {
    uint32_t mb = 0;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      x[z][e] = __fmul_rn(x[z][e], p.cb);  // (exact for b = 1: c_b = 1)
      mb = max(mb, __float_as_uint(fabsf(x[z][e])));  // ordered as the values
    }
    s[z] = __fdiv_rn(__uint_as_float(__reduce_max_sync(kFull, mb)), 127.0f);
  }
#pragma unroll
  for (int z = 0; z < kBatch; z++) {
    // c = rint(fl(x / s)) without dividing: t = fl(x fl(1/s)) is within 127 * 3 * 2^-24 < 2^-15 of
    // the quotient and of its rounding, so rint(t) is rint of it unless t is that near to a half
    // (then divide).  The low byte of t + 1.5 * 2^23 is rint(t) in two's complement.
    const float r = s[z] > 0.0f ? __frcp_rn(s[z]) : 0.0f;
    uint32_t cb[4];
    float far = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const float t = __fmul_rn(x[z][e], r), m = __fadd_rn(t, kMagic);
      far = fmaxf(far, fabsf(__fsub_rn(t, __fsub_rn(m, kMagic))));
      cb[e] = __float_as_uint(m);
    }
    if (far > 0.5f - 0x1p-15f) {
#pragma unroll
      for (int e = 0; e < 4; e++) cb[e] = __float_as_uint(__fadd_rn(rintf(__fdiv_rn(x[z][e], s[z])), kMagic));
    }
    const int i = i0 + z * kWarps;
    if (i < nrow) {
      const uint32_t code = prmt(prmt(cb[0], cb[1], 0x0040u), prmt(cb[2], cb[3], 0x0040u), 0x5410u);
      const uint32_t sign = prmt(code, code, 0xBA98u);  // 0xFF in the bytes of negative codes
      uint32_t* const tile = frag + (i >> 4) * (16 * kRowBytes / 4);
      put_codes(tile, i & 15, lane, code & sign);
      put_codes(tile, i & 15, 32 + lane, code & ~sign);
      if (lane == 0) sq[i] = s[z];
    }
  }
}

template <int G, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(SelectParams p) {
  // A cluster's few queries take each instruction once: less code there (fewer fetches), more of it
  // in flight at a time where there are many (decode 12.0 us instead of 13.7, a chunk 36.5 instead
  // of 37.8).
  constexpr int kBatch = CLUSTER ? 2 : 4, kLoads = CLUSTER ? 2 : 4;
  griddep_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int red[2][2][kWarps];
  __shared__ __align__(16) int hist[kWarps][kBins];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const uint32_t C = CLUSTER ? cluster_size() : 1u, rank = CLUSTER ? cluster_rank() : 0u;
  const int item = blockIdx.x / C, h = blockIdx.y;
  const int Q = p.queries, KW = key_stride(p.max_pages_per_seq);
  uint32_t* const keys = reinterpret_cast<uint32_t*>(smem);              // [Q][KW]
  uint32_t* const frag = keys + static_cast<size_t>(Q) * KW;             // [rows / 16] MMA tiles of 16 query heads
  float* const sq = reinterpret_cast<float*>(frag + tile_rows(Q, G) * (kRowBytes / 4));
  griddep_wait();
  // The tile's queries t0 .. t0 + nq - 1 of sequence b.  Tile slots as in the bounds kernel:
  // sequence b has those from cu[b] / Q + b on, at least ceil(n / Q) of them.
  int b = item, t0 = item, nq = 1, n = 1, i0 = 0;
  if (p.cu_q) {
    auto slot0 = [&](int s) { return __ldg(p.cu_q + s) / Q + s; };
    b = warp_find(p.batch, item, slot0);
    const int first = __ldg(p.cu_q + b);
    n = __ldg(p.cu_q + b + 1) - first;
    i0 = (item - slot0(b)) * Q;
    nq = min(Q, n - i0);
    t0 = first + i0;
    // (the whole cluster leaves: it shares the item)
    if (nq <= 0 || i0 < 0 || t0 < 0 || t0 + nq > p.total_q) return;
  }
  const int L = __ldg(p.seq_lens + b);
  const bool bad = L < 0 || static_cast<long long>(L) > (static_cast<long long>(p.max_pages_per_seq) << p.page_shift) ||
                   (p.cu_q && n > L);
  if (bad && tid == 0 && rank == 0) atomicOr(p.status, KVQ_DEV_BAD_POS_BIT);
  // Pages of query i: those that start at or before its position L - n + i0 + i.
  const int pos0 = bad ? -1 : L - n + i0;
  auto pages_of = [&](int i) { return bad || pos0 + i < 0 ? 0 : ((pos0 + i) >> p.page_shift) + 1; };
  const int nmax = pages_of(nq - 1);
  const int k = p.num_blocks;

  // No query of the tile has a choice to make: skip the scores.
  const bool choose = nmax > k;
  if (choose) {
    const int nrow = tile_rows(nq, G);
    const int g = lane >> 2, c = lane & 3;
    const int ntile = (nmax + kTilePages - 1) / kTilePages, step = kWarps * static_cast<int>(C);
    const int32_t* table = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;
    const __half* qt = p.q + (static_cast<size_t>(t0) * p.num_kv_heads + h) * G * kD;
    // Row i of the MMA tiles: heads 2 x and 2 x + 1 of a query in rows R and R + 8 (G = 1: a query
    // each).
    constexpr int kPairs = G > 1 ? G / 2 : 1;
    auto query_of = [&](int i) { return G == 1 ? i : (i >> 4) * (16 / G) + (i & 7) / kPairs; };
    auto load_q = [&](uint2 (&raw)[kBatch], int i0) {
#pragma unroll
      for (int z = 0; z < kBatch; z++) {
        const int i = i0 + z * kWarps, q = query_of(i);
        const int head = G == 1 ? 0 : 2 * ((i & 7) % kPairs) + ((i >> 3) & 1);
        raw[z] = make_uint2(0u, 0u);
        if (i < nrow && q < nq)
          raw[z] = __ldcg(reinterpret_cast<const uint2*>(qt + (static_cast<size_t>(q) * p.num_kv_heads * G + head) * kD) + lane);
      }
    };
    // The first q rows are in flight first of all, then the first step's page rows.
    uint2 raw[kBatch];
    load_q(raw, w);
    constexpr int kN = kTilePages / 8;
    u32x8 rows[kN][2];
    float sigma[kN];  // of page g of MMA tile r (0: no page there, or a bad one)
    int pid[kN];  // page g of MMA tile r, a step ahead of the rows
    auto load_ids = [&](int mt) {
#pragma unroll
      for (int r = 0; r < kN; r++) {
        const int lp = mt * kTilePages + 8 * r + g;
        pid[r] = lp < nmax ? __ldg(table + lp) : -1;
      }
    };
    auto load_rows = [&](int mt) {
#pragma unroll
      for (int r = 0; r < kN; r++) {
        const bool none = pid[r] < 0 || pid[r] >= p.num_pages;
        if (none && mt * kTilePages + 8 * r + g < nmax && c == 0) atomicOr(p.status, KVQ_DEV_BAD_PAGE_BIT);
        const size_t row = static_cast<size_t>(none ? 0 : pid[r]) * p.num_kv_heads + h;
        const int8_t* src = p.codes + row * (2 * kD) + 32 * c;
        rows[r][0] = ldg_256(src);
        rows[r][1] = ldg_256(src + 128);
        sigma[r] = none ? 0.0f : __ldcg(p.scale + row);
      }
    };
    int mt = static_cast<int>(rank) * kWarps + w;
    load_ids(mt);
    if (mt < ntile) load_rows(mt);
    load_ids(mt + step);

#pragma unroll 1
    for (int i0 = w; i0 < nrow; i0 += kBatch * kWarps) {
      if (i0 != w) load_q(raw, i0);
      prep_rows<kBatch>(raw, frag, sq, i0, nrow, lane, p);
    }
    // Keys past the last scored tile of pages count for nothing.
    if (rank == 0) {
      const int from = ntile * kTilePages, to = key_words(nmax);
      for (int q = 0; q < nq; q++)
        for (int i = from + tid; i < to; i += kThreads) keys[q * KW + i] = 0u;
    }
    if (CLUSTER) cluster_sync();  // every CTA of the cluster runs before its memory is written
    else __syncthreads();

    const uint32_t keys0 = CLUSTER ? map_rank(smem_addr(keys), 0) : smem_addr(keys);
    const uint32_t frag_s = smem_addr(frag);
    for (; mt < ntile; mt += step) {
      // Sigma of this lane's output pages: 8 r + 2 c and 8 r + 2 c + 1 of the tile.
      float sg[kN][2];
#pragma unroll
      for (int r = 0; r < kN; r++) {
        sg[r][0] = __shfl_sync(kFull, sigma[r], 8 * c);
        sg[r][1] = __shfl_sync(kFull, sigma[r], 8 * c + 4);
      }
      // Keys of n pages of query q, then their stores (the keys' chains interleave).
      auto put = [&](int q, const auto& lp, const auto& v, const auto& factor) {
        constexpr int kPut = sizeof(lp) / sizeof(int);
        const unsigned span = static_cast<unsigned>(max(pages_of(q) - p.recent - p.sink, 0));
        uint32_t key[kPut];
#pragma unroll
        for (int i = 0; i < kPut; i++) {
          key[i] = ordered(v[i], factor[i]);
          // (always taken, or behind the query: one unsigned comparison for both ends)
          if (static_cast<unsigned>(lp[i] - p.sink) >= span) key[i] = 0u;
        }
        if (q >= nq) return;
        const uint32_t dst = keys0 + static_cast<uint32_t>(q * KW) * 4;
#pragma unroll
        for (int i = 0; i < kPut; i++) {
          if (CLUSTER) st_cluster(dst + lp[i] * 4, key[i]);
          else sts_32(dst + lp[i] * 4, key[i]);
        }
      };
#pragma unroll 1
      for (int j = 0; j < nrow / 16; j++) {
        // Sums start at the integer of 1.5 * 2^23: their bits are then the float 1.5 * 2^23 + I.
        int acc[kN][4];
#pragma unroll
        for (int r = 0; r < kN; r++)
#pragma unroll
          for (int e = 0; e < 4; e++) acc[r][e] = kMagicBits;
        const uint32_t fr = frag_s + (j * 8 * 32 + lane) * 16;
#pragma unroll
        for (int s = 0; s < 8; s++) {
          const uint4 f = lds_128(fr + s * 512);
#pragma unroll
          for (int r = 0; r < kN; r++)
            mma_16832_s8(acc[r], f.x, f.y, f.z, f.w, rows[r][s >> 2].w[2 * (s & 3)], rows[r][s >> 2].w[2 * (s & 3) + 1]);
        }
        // Rows g (acc 0, 1) and g + 8 (acc 2, 3) of pages 8 r + 2 c, + 1, times the heads' factors.
        const float s0 = sq[16 * j + g], s1 = sq[16 * j + 8 + g];
        const uint64_t S0 = f2_pack(s0, s0), S1 = f2_pack(s1, s1), MM = f2_pack(kMagic, kMagic);
        const int lp0 = mt * kTilePages + 2 * c;
        const int odd = g & 1, high = (g >> 1) & 1;
        float v[kN][4];
#pragma unroll
        for (int r = 0; r < kN; r++)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const uint64_t d = f2_sub(f2_pack(__int_as_float(acc[r][e]), __int_as_float(acc[r][e + 1])), MM);
            const float2 w2 = f2_unpack(f2_mul(d, e ? S1 : S0));
            v[r][e] = w2.x;
            v[r][e + 1] = w2.y;
          }
        if constexpr (G <= 2) {
          // Every lane stores all its pages: of rows g and g + 8 (G = 1), or of their maximum.
#pragma unroll
          for (int x = 0; x < 2; x++) {
            if (G == 2 && x) break;
            int lp[2 * kN];
            float u[2 * kN], f[2 * kN];
#pragma unroll
            for (int r = 0; r < kN; r++)
#pragma unroll
              for (int e = 0; e < 2; e++) {
                lp[2 * r + e] = lp0 + 8 * r + e;
                u[2 * r + e] = G == 2 ? fmaxf(v[r][e], v[r][2 + e]) : v[r][2 * x + e];
                f[2 * r + e] = sg[r][e];
              }
            put(G == 2 ? 8 * j + g : 16 * j + 8 * x + g, lp, u, f);
          }
        } else {
          // Lanes g and g ^ 1 share a query: the odd one keeps the odd pages.
          float t[kN], f[kN];
#pragma unroll
          for (int r = 0; r < kN; r++) {
            const float u0 = fmaxf(v[r][0], v[r][2]), u1 = fmaxf(v[r][1], v[r][3]);
            t[r] = fmaxf(odd ? u1 : u0, __shfl_xor_sync(kFull, odd ? u0 : u1, 4));
            f[r] = odd ? sg[r][1] : sg[r][0];
          }
          if constexpr (G == 4) {
            int lp[kN];
#pragma unroll
            for (int r = 0; r < kN; r++) lp[r] = lp0 + 8 * r + odd;
            put(4 * j + (g >> 1), lp, t, f);
          } else {
            // ... and g ^ 2: the one with that bit set keeps the second of two MMA tiles.
            int lp[kN / 2];
            float u[kN / 2], fh[kN / 2];
#pragma unroll
            for (int r = 0; r < kN / 2; r++) {
              const float far = __shfl_xor_sync(kFull, high ? t[2 * r] : t[2 * r + 1], 8);
              u[r] = fmaxf(high ? t[2 * r + 1] : t[2 * r], far);
              fh[r] = high ? f[2 * r + 1] : f[2 * r];
              lp[r] = lp0 + 16 * r + (high ? 8 : 0) + odd;
            }
            put(2 * j + (g >> 2), lp, u, fh);
          }
        }
      }
      if (mt + step < ntile) {
        load_rows(mt + step);
        load_ids(mt + 2 * step);
      }
    }
    if (CLUSTER) cluster_sync();
    else __syncthreads();
  }
  if (rank != 0) return;

  // Teams of TW warps share a query (TW a power of two, all warps for one query).
  int TW = 1;
  while (TW * 2 * nq <= kWarps) TW *= 2;
  const int team = w / TW, tw = w - team * TW;
  int parity = 0;
  auto team_sync = [&]() {
    if (TW > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * TW) : "memory");
    else __syncwarp();
  };
  // Two values per warp, exchanged in the team: f(i, a, b) for its warps i.  The two buffers
  // alternate, so one barrier per exchange is enough.
  auto exchange = [&](uint32_t a, uint32_t b, auto&& f) {
    if (lane == 0) {
      red[parity][0][w] = static_cast<int>(a);
      red[parity][1][w] = static_cast<int>(b);
    }
    team_sync();
    for (int i = 0; i < TW; i++)
      f(i, static_cast<uint32_t>(red[parity][0][team * TW + i]), static_cast<uint32_t>(red[parity][1][team * TW + i]));
    parity ^= 1;
  };
  int* const bins = hist[team * TW];
  const uint32_t bins_s = smem_addr(bins);
  for (int q = team; q < nq; q += kWarps / TW) {
    const int np = pages_of(q);
    int32_t* out = p.blocks + (static_cast<size_t>(t0 + q) * p.num_kv_heads + h) * k;
    if (np <= k) {
      for (int i = tw * 32 + lane; i < k; i += 32 * TW) out[i] = i < np ? i : -1;
      continue;
    }
    const uint32_t* kq = keys + q * KW;
    const uint4* kq4 = reinterpret_cast<const uint4*>(kq);
    const int words4 = key_words(np) / 4;
    // f on this team's share of the keys, kLoads loads in flight.
    auto each4 = [&](auto&& f) {
      for (int i = tw * 32 + lane; i < words4; i += kLoads * 32 * TW) {
        uint4 v[kLoads];
#pragma unroll
        for (int z = 0; z < kLoads; z++)
          v[z] = i + z * 32 * TW < words4 ? kq4[i + z * 32 * TW] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int z = 0; z < kLoads; z++) f(v[z]);
      }
    };
    // Taken: the pages that always are, the keys >= T, and the first `quota` keys equal to T - 1.
    // (Of a query without a score every key may be the largest integer, NaN's: T is then 0, one
    // more than it, and no key is above.)
    uint32_t T = 0xFFFFFFFFu;
    int quota = 0;
    const int chosen = k - p.sink - p.recent;  // >= 0 (host-checked), < the keys that are a choice
    int need = chosen;
    if (need > 0) {
      uint32_t lo = 0xFFFFFFFFu, hi = 0u;
      each4([&](uint4 v) {
        lo = min(min(min(lo, v.x - 1u), min(v.y - 1u, v.z - 1u)), v.w - 1u);  // (0 becomes the largest)
        hi = max(max(max(hi, v.x), max(v.y, v.z)), v.w);
      });
      lo = __reduce_min_sync(kFull, lo);
      hi = __reduce_max_sync(kFull, hi);
      if (TW > 1) exchange(lo, hi, [&](int, uint32_t a, uint32_t b2) {
        lo = min(lo, a);
        hi = max(hi, b2);
      });
      lo += 1u;
      while (true) {
        // [lo, hi] in bins of 2^sh keys.
        const uint32_t width = hi - lo;
        const int sh = width < kBins ? 0 : 24 - __clz(width);
        for (int i = tw * 32 + lane; i < kBins; i += 32 * TW) bins[i] = 0;
        team_sync();
        each4([&](uint4 v) {
          const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int z = 0; z < 4; z++) count_if(bins_s + ((e[z] - lo) >> sh) * 4, e[z] - lo <= width);
        });
        team_sync();
        // Bins from the top: lane j holds bins 255 - 8 j .. 248 - 8 j.
        int cnt[8], sum = 0;
        const int4* b4 = reinterpret_cast<const int4*>(bins) + 62 - 2 * lane;
        const int4 u0 = b4[1], u1 = b4[0];
        cnt[0] = u0.w, cnt[1] = u0.z, cnt[2] = u0.y, cnt[3] = u0.x;
        cnt[4] = u1.w, cnt[5] = u1.z, cnt[6] = u1.y, cnt[7] = u1.x;
#pragma unroll
        for (int i = 0; i < 8; i++) sum += cnt[i];
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int y = __shfl_up_sync(kFull, incl, d);
          if (lane >= d) incl += y;
        }
        const int src = __ffs(__ballot_sync(kFull, incl >= need)) - 1;
        int above = incl - sum, bin = 0, inbin = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          if (inbin == 0 && above + cnt[i] >= need) {
            bin = 255 - 8 * lane - i;
            inbin = cnt[i];
          }
          if (inbin == 0) above += cnt[i];
        }
        above = __shfl_sync(kFull, above, src);
        bin = __shfl_sync(kFull, bin, src);
        inbin = __shfl_sync(kFull, inbin, src);
        team_sync();  // the bins are read: the next round may clear them
        need -= above;
        lo += static_cast<uint32_t>(bin) << sh;
        if (inbin == need) {
          T = lo;
          break;
        }
        if (sh == 0) {
          T = lo + 1u;
          quota = need;
          break;
        }
        hi = lo + min(hi - lo, (1u << sh) - 1u);
        if (inbin <= 32) {
          // Few keys are left: collect them, a lane each, and rank them against one another.
          if (tw == 0) bins[lane] = 0;
          if (tw == 0 && lane == 0) bins[32] = 0;
          team_sync();
          const uint32_t span = hi - lo;
          each4([&](uint4 v) {
            const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int z = 0; z < 4; z++)
              if (e[z] - lo <= span) bins[atomicAdd(bins + 32, 1)] = static_cast<int>(e[z]);
          });
          team_sync();
          const uint32_t mine = static_cast<uint32_t>(bins[lane]);  // 0: none
          int higher = 0, same = 0;
          for (int i = 0; i < inbin; i++) {
            const uint32_t other = __shfl_sync(kFull, mine, i);
            higher += other > mine;
            same += other == mine;
          }
          const bool it = lane < inbin && higher < need && higher + same >= need;
          const int src2 = __ffs(__ballot_sync(kFull, it)) - 1;
          T = __shfl_sync(kFull, mine, src2);
          higher = __shfl_sync(kFull, higher, src2);
          same = __shfl_sync(kFull, same, src2);
          team_sync();  // the list is read
          if (higher + same != need) {
            quota = need - higher;
            T += 1u;
          }
          break;
        }
      }
    }
    const bool any_above = chosen > 0 && T != 0u;
    // The pages in ascending order: each warp of the team a contiguous part; lane i of a warp
    // holds the mask of the part's pages 32 i .. 32 i + 31.
    const int words = (np + 31) / 32, per = (words + TW - 1) / TW;
    const int w0 = tw * per, w1 = min(words, w0 + per);
    auto masks = [&](int base, uint32_t& sure, uint32_t& tie) {
      // Bits of the pages below `sink` and from np - recent to np.
      auto up_to = [&](int n) {  // bits of the lane's word that are pages below n
        const int m = n - (base + lane) * 32;
        return m >= 32 ? 0xFFFFFFFFu : m <= 0 ? 0u : (1u << m) - 1u;
      };
      uint32_t forced = 0;
      if (base + lane < w1) forced = up_to(p.sink) | (up_to(np) & ~up_to(np - p.recent));
      sure = tie = 0;
      const int m = min(32, w1 - base);
#pragma unroll 8
      for (int i = 0; i < m; i++) {
        const uint32_t key = kq[(base + i) * 32 + lane];
        const uint32_t ms = __ballot_sync(kFull, key >= T && any_above);
        if (lane == i) sure = ms;
      }
      sure |= forced;
      if (quota) {
        for (int i = 0; i < m; i++) {
          const uint32_t mt = __ballot_sync(kFull, kq[(base + i) * 32 + lane] == T - 1u);
          if (lane == i) tie = mt;
        }
      }
    };
    // Once to count what the team's earlier warps take (when there are any), once to write.
    int before = 0, ties = 0;  // sure and tied pages of the team's earlier warps
#pragma unroll 1
    for (int pass = TW > 1 ? 0 : 1; pass < 2; pass++) {
      int cs = 0, ct = 0;
#pragma unroll 1
      for (int base = w0; base < w1; base += 32) {
        uint32_t sure, tie;
        masks(base, sure, tie);
        // Inclusive prefixes over the lanes: sure pages low, tied pages high (both below 2^16 in a
        // step of 1024 pages).
        const int mine = __popc(sure) | (__popc(tie) << 16);
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int y = __shfl_up_sync(kFull, incl, d);
          if (lane >= d) incl += y;
        }
        const int total = __shfl_sync(kFull, incl, 31);
        if (pass) {
          const int es = before + cs + ((incl - mine) & 0xFFFF), et = ties + ct + ((incl - mine) >> 16);
          int at = es + min(et, quota), left = quota - et;  // tied pages still to take
          for (uint32_t m = sure | tie; m; m &= m - 1u) {
            const int bit = __ffs(m) - 1;
            if ((tie >> bit) & 1u && left-- <= 0) continue;
            if (at < k) out[at++] = (base + lane) * 32 + bit;
          }
        }
        cs += total & 0xFFFF;
        ct += total >> 16;
      }
      if (pass == 0) exchange(cs, ct, [&](int i, uint32_t a, uint32_t b2) {
        if (i < tw) {
          before += static_cast<int>(a);
          ties += static_cast<int>(b2);
        }
      });
    }
  }
}

template <int G, bool CLUSTER>
int launch_kernel(cudaLaunchConfig_t& cfg, const SelectParams& p) {
  if (!ensure_smem<select_kernel<G, CLUSTER>>(kSmemCap)) return -2;
  return cudaLaunchKernelEx(&cfg, select_kernel<G, CLUSTER>, p) == cudaSuccess ? 0 : -2;
}

template <int G>
int launch_one(cudaLaunchConfig_t& cfg, const SelectParams& p) {
  return cfg.numAttrs > 1 ? launch_kernel<G, true>(cfg, p) : launch_kernel<G, false>(cfg, p);
}

}  // namespace

int launch_select(SelectParams p, int num_sms, cudaStream_t stream) {
  if (p.total_q == 0) return 0;
  if (select_smem(1, p.group, p.max_pages_per_seq) > kSmemCap) return -1;
  if (p.num_kv_heads > 65535) return -1;
  // Queries of a tile: as many as leave a CTA per SM and two CTAs' keys in an SM's memory.
  int Q = p.cu_q ? kMaxQueries : 1;
  auto tiles = [&](int q) {
    return (p.cu_q ? static_cast<long long>(p.total_q) / q + p.batch : p.batch) * p.num_kv_heads;
  };
  while (Q > 1 && (select_smem(Q, p.group, p.max_pages_per_seq) > 104 * 1024 || tiles(Q) < num_sms)) Q /= 2;
  p.queries = Q;
  // CTAs that share a tile's pages: while the grid has room for them and every warp keeps a step.
  const int ptiles = (p.max_pages_per_seq + kTilePages - 1) / kTilePages;
  int C = 1;
  while (C < kMaxCluster && tiles(Q) * C * 2 <= 2 * num_sms && ptiles >= 2 * kWarps * C) C *= 2;
  const long long items = tiles(Q) / p.num_kv_heads;
  if (items * C > 0x7fffffffLL) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * C), static_cast<unsigned>(p.num_kv_heads));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = select_smem(Q, p.group, p.max_pages_per_seq);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  switch (p.group) {
    case 1: return launch_one<1>(cfg, p);
    case 2: return launch_one<2>(cfg, p);
    case 4: return launch_one<4>(cfg, p);
    case 8: return launch_one<8>(cfg, p);
    default: return -1;
  }
}

}  // namespace kvq
