// block_select.cu -- the pages that each query and KV head attends, chosen by an upper bound of
// q.k over the page's keys, for sm_100a.
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
// Scores.  I is a product of the page rows (256 int8: lo, then hi) with the columns of all query
// heads of a tile (256 int8: min(c, 0), then max(c, 0)): mma.sync m16n8k32 s8 with 16 pages as
// the M side, read from global memory straight into fragments (a row's 64-byte pieces are whole
// sectors; a dot product does not depend on the order of its terms, so lane c of a quad takes
// bytes 64 i + 16 c on).  The scores of a tile's queries over all pages stay in shared memory.
//
// Choice.  Keys are the scores as ordered 32-bit integers; the k-th largest is found by bisection
// between the smallest and the largest key, which ends as soon as a threshold leaves exactly k
// keys, then the pages are written in ascending order by ballots.  A team of warps shares a query.
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
constexpr int kMaxQueries = 8;                 // queries of a tile
constexpr int kColStride = 2 * kD + 16;        // bytes of a column of q codes (bank spread)
constexpr int kMaxCluster = 8;
constexpr unsigned kFull = 0xffffffffu;

__host__ __device__ inline int key_words(int pages) { return (pages + 127) / 128 * 128; }

__host__ __device__ inline int tile_columns(int queries, int group) { return (queries * group + 7) / 8 * 8; }

inline size_t select_smem(int queries, int group, int pages) {
  return static_cast<size_t>(queries) * key_words(pages) * 4 + tile_columns(queries, group) * (kColStride + 4);
}

constexpr size_t kSmemCap = 200 * 1024;

// Float -> integer of the same order; never 0 (0 marks pages that are not a choice).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 -> +0
  const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
  return k ? k : 1u;
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

// One query head's int8 codes into its column (and its factor), by one warp.
__device__ __forceinline__ void prep_column(const __half* row, uint8_t* col, float* sq, int lane,
                                            const SelectParams& p) {
  const uint2 raw = __ldg(reinterpret_cast<const uint2*>(row) + lane);  // channels 4 lane ..
  const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
  const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
  float x[4] = {lo.x, lo.y, hi.x, hi.y};
  if (p.hadamard_block > 1) {
    const float a0 = __fadd_rn(x[0], x[1]), a1 = __fsub_rn(x[0], x[1]);
    const float a2 = __fadd_rn(x[2], x[3]), a3 = __fsub_rn(x[2], x[3]);
    x[0] = __fadd_rn(a0, a2);
    x[2] = __fsub_rn(a0, a2);
    x[1] = __fadd_rn(a1, a3);
    x[3] = __fsub_rn(a1, a3);
#pragma unroll
    for (int s = 0; s < 5; s++) {
      if ((4 << s) < p.hadamard_block) {
        const float sgn = ((lane >> s) & 1) ? -1.0f : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = __fmaf_rn(x[e], sgn, __shfl_xor_sync(kFull, x[e], 1 << s));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; e++) x[e] = __fmul_rn(x[e], p.cb);
  }
  float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
  for (int d = 1; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
  const float s = __fdiv_rn(m, 127.0f);
  uint32_t neg = 0, pos = 0;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const int c = s > 0.0f ? static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(x[e], s)), -127.0f), 127.0f)) : 0;
    neg |= (static_cast<uint32_t>(min(c, 0)) & 0xFFu) << (8 * e);
    pos |= (static_cast<uint32_t>(max(c, 0)) & 0xFFu) << (8 * e);
  }
  reinterpret_cast<uint32_t*>(col)[lane] = neg;
  reinterpret_cast<uint32_t*>(col)[32 + lane] = pos;
  if (lane == 0) *sq = s;
}

template <int G>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(SelectParams p) {
  griddep_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int red[2][2][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const uint32_t C = cluster_size(), rank = cluster_rank();
  const int item = blockIdx.x / C, h = blockIdx.y;
  const int Q = p.queries, KW = key_words(p.max_pages_per_seq);
  uint32_t* const keys = reinterpret_cast<uint32_t*>(smem);              // [Q][KW]
  uint8_t* const cols = smem + static_cast<size_t>(Q) * KW * 4;          // [columns][kColStride]
  float* const sq = reinterpret_cast<float*>(cols + tile_columns(Q, G) * kColStride);
  griddep_wait();
  // The tile's queries t0 .. t0 + nq - 1 of sequence b.  Tile slots as in the bounds kernel:
  // sequence b has those from cu[b] / Q + b on, at least ceil(n / Q) of them.
  int b = item, t0 = item, nq = 1, n = 1, i0 = 0;
  if (p.cu_q) {
    auto slot0 = [&](int s) { return __ldg(p.cu_q + s) / Q + s; };
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (slot0(mid) <= item) lo = mid; else hi = mid;
    }
    b = lo;
    const int first = __ldg(p.cu_q + b);
    n = __ldg(p.cu_q + b + 1) - first;
    i0 = (item - slot0(b)) * Q;
    nq = min(Q, n - i0);
    t0 = first + i0;
    // (the whole cluster leaves: it shares the item)
    if (nq <= 0 || i0 < 0 || t0 < 0 || t0 + nq > p.total_q) return;
  }
  const int S = p.page_size, L = __ldg(p.seq_lens + b);
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
    const int ncol = nq * G, ncolp = (ncol + 7) / 8 * 8;
    const __half* qt = p.q + (static_cast<size_t>(t0) * p.num_kv_heads + h) * G * kD;
    for (int c = w; c < ncolp; c += kWarps) {
      if (c < ncol) {
        prep_column(qt + (static_cast<size_t>(c / G) * p.num_kv_heads * G + c % G) * kD, cols + c * kColStride, sq + c,
                    lane, p);
      } else {
        reinterpret_cast<uint32_t*>(cols + c * kColStride)[lane] = 0u;
        reinterpret_cast<uint32_t*>(cols + c * kColStride)[32 + lane] = 0u;
        if (lane == 0) sq[c] = 0.0f;
      }
    }
    // Keys past the last scored tile of pages count for nothing.
    if (rank == 0) {
      const int from = (nmax + 15) / 16 * 16, to = key_words(nmax);
      for (int q = 0; q < nq; q++)
        for (int i = from + tid; i < to; i += kThreads) keys[q * KW + i] = 0u;
    }
    if (C > 1) cluster_sync();  // every CTA of the cluster runs before its memory is written
    else __syncthreads();

    const int g = lane >> 2, c = lane & 3;
    const uint32_t keys0 = C > 1 ? map_rank(smem_addr(keys), 0) : smem_addr(keys);
    const int ntile = (nmax + 15) / 16, step = kWarps * static_cast<int>(C);
    const int32_t* table = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;
    for (int mt = static_cast<int>(rank) * kWarps + w; mt < ntile; mt += step) {
      uint4 a[2][4];
      float sg[2];
      bool pad[2];
#pragma unroll
      for (int r = 0; r < 2; r++) {
        const int lp = mt * 16 + g + 8 * r;
        int page = lp < nmax ? __ldg(table + lp) : -1;
        pad[r] = page < 0 || page >= p.num_pages;
        if (pad[r] && lp < nmax && c == 0) atomicOr(p.status, KVQ_DEV_BAD_PAGE_BIT);
        const size_t row = static_cast<size_t>(pad[r] ? 0 : page) * p.num_kv_heads + h;
        const uint4* src = reinterpret_cast<const uint4*>(p.codes + row * (2 * kD)) + c;
#pragma unroll
        for (int i = 0; i < 4; i++) a[r][i] = __ldg(src + 4 * i);
        sg[r] = __ldg(p.scale + row);
      }
      for (int j = 0; j < ncolp / 8; j++) {
        int acc[4] = {0, 0, 0, 0};
        const uint4* bc = reinterpret_cast<const uint4*>(cols + (8 * j + g) * kColStride) + c;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const uint4 bb = bc[4 * i];
          mma_16832_s8(acc, a[0][i].x, a[1][i].x, a[0][i].y, a[1][i].y, bb.x, bb.y);
          mma_16832_s8(acc, a[0][i].z, a[1][i].z, a[0][i].w, a[1][i].w, bb.z, bb.w);
        }
        // Columns 2c, 2c + 1 of row g (acc 0, 1) and g + 8 (acc 2, 3).
        const float s0 = sq[8 * j + 2 * c], s1 = sq[8 * j + 2 * c + 1];
#pragma unroll
        for (int r = 0; r < 2; r++) {
          float v0 = __fmul_rn(static_cast<float>(acc[2 * r]), s0), v1 = __fmul_rn(static_cast<float>(acc[2 * r + 1]), s1);
          const int lp = mt * 16 + g + 8 * r;
          auto put = [&](int q, float v) {
            if (q >= nq) return;
            const int np = pages_of(q);
            uint32_t key = pad[r] ? 1u : ordered(__fmul_rn(v, sg[r]));
            if (lp < p.sink || lp >= np - p.recent) key = 0u;  // always taken, or past the query
            const uint32_t dst = keys0 + static_cast<uint32_t>(q * KW + lp) * 4;
            if (C > 1) st_cluster(dst, key);
            else sts_32(dst, key);
          };
          if constexpr (G == 1) {
            put(8 * j + 2 * c, v0);
            put(8 * j + 2 * c + 1, v1);
          } else {
            v0 = fmaxf(v0, v1);
            if constexpr (G >= 4) v0 = fmaxf(v0, __shfl_xor_sync(kFull, v0, 1));
            if constexpr (G == 8) v0 = fmaxf(v0, __shfl_xor_sync(kFull, v0, 2));
            if (c % (G / 2) == 0) put((8 * j + 2 * c) / G, v0);
          }
        }
      }
    }
    if (C > 1) cluster_sync();
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
  };
  // Sum over the team; the two buffers alternate, so one barrier per sum is enough.
  auto team_sum = [&](int v) {
    v = __reduce_add_sync(kFull, v);
    if (TW == 1) return v;
    if (lane == 0) red[parity][0][w] = v;
    team_sync();
    int s = 0;
    for (int i = 0; i < TW; i++) s += red[parity][0][team * TW + i];
    parity ^= 1;
    return s;
  };
  for (int q = team; q < nq; q += kWarps / TW) {
    const int np = pages_of(q);
    int32_t* out = p.blocks + (static_cast<size_t>(t0 + q) * p.num_kv_heads + h) * k;
    if (np <= k) {
      for (int i = tw * 32 + lane; i < k; i += 32 * TW) out[i] = i < np ? i : -1;
      continue;
    }
    const int want = k - p.sink - p.recent;  // >= 0 (host-checked)
    const uint32_t* kq = keys + q * KW;
    const uint4* kq4 = reinterpret_cast<const uint4*>(kq);
    const int words4 = key_words(np) / 4;
    // Threshold T: the keys >= T are `want`, or more than that with too few keys >= T + 1.
    uint32_t T = 0xFFFFFFFFu;
    int over = 0;  // keys above T
    bool exact = true;  // exactly `want` keys >= T
    if (want > 0) {
      uint32_t kmin = 0xFFFFFFFFu, kmax = 0u;
      for (int i = tw * 32 + lane; i < words4; i += 32 * TW) {
        const uint4 v = kq4[i];
        const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int z = 0; z < 4; z++) {
          kmax = max(kmax, e[z]);
          if (e[z]) kmin = min(kmin, e[z]);
        }
      }
      kmin = __reduce_min_sync(kFull, kmin);
      kmax = __reduce_max_sync(kFull, kmax);
      if (TW > 1) {
        if (lane == 0) {
          red[parity][0][w] = static_cast<int>(kmin);
          red[parity][1][w] = static_cast<int>(kmax);
        }
        team_sync();
        for (int i = 0; i < TW; i++) {
          kmin = min(kmin, static_cast<uint32_t>(red[parity][0][team * TW + i]));
          kmax = max(kmax, static_cast<uint32_t>(red[parity][1][team * TW + i]));
        }
        parity ^= 1;
      }
      // count(>= lo) > want, or lo = kmin; count(>= hi) < want; 64-bit for hi = kmax + 1.
      unsigned long long lo = kmin, hi = static_cast<unsigned long long>(kmax) + 1;
      exact = false;
      while (hi - lo > 1) {
        const uint32_t mid = static_cast<uint32_t>((lo + hi) >> 1);
        int cnt = 0;
        for (int i = tw * 32 + lane; i < words4; i += 32 * TW) {
          const uint4 v = kq4[i];
          cnt += (v.x >= mid) + (v.y >= mid) + (v.z >= mid) + (v.w >= mid);
        }
        cnt = team_sum(cnt);
        if (cnt == want) {
          lo = mid;
          exact = true;
          break;
        }
        if (cnt > want) lo = mid;
        else {
          hi = mid;
          over = cnt;
        }
      }
      T = static_cast<uint32_t>(lo);
    }
    // The pages in ascending order: each warp of the team a contiguous part, 32 pages a step.
    const int steps = (np + 31) / 32, per = (steps + TW - 1) / TW;
    const int s0 = tw * per, s1 = min(steps, s0 + per);
    auto flags = [&](int i, bool& sure, bool& tie) {
      const uint32_t key = i < np ? kq[i] : 0u;
      const bool forced = i < np && (i < p.sink || i >= np - p.recent);
      sure = forced || (want > 0 && key != 0u && (exact ? key >= T : key > T));
      tie = !exact && want > 0 && !forced && key == T;
    };
    int before = 0, ties = 0;  // sure and tied pages of the team's earlier warps
    if (TW > 1) {
      int cs = 0, ct = 0;
      for (int s = s0; s < s1; s++) {
        bool sure, tie;
        flags(s * 32 + lane, sure, tie);
        cs += __popc(__ballot_sync(kFull, sure));
        ct += __popc(__ballot_sync(kFull, tie));
      }
      if (lane == 0) {
        red[parity][0][w] = cs;
        red[parity][1][w] = ct;
      }
      team_sync();
      for (int i = 0; i < tw; i++) {
        before += red[parity][0][team * TW + i];
        ties += red[parity][1][team * TW + i];
      }
      parity ^= 1;
    }
    const int quota = want - over;  // tied pages to take
    const unsigned below = (1u << lane) - 1u;
    for (int s = s0; s < s1; s++) {
      bool sure, tie;
      flags(s * 32 + lane, sure, tie);
      const unsigned ms = __ballot_sync(kFull, sure), mt = __ballot_sync(kFull, tie);
      const bool take = sure || (tie && ties + __popc(mt & below) < quota);
      if (take) {
        const int at = before + __popc(ms & below) + min(ties + __popc(mt & below), quota);
        if (at < k) out[at] = s * 32 + lane;
      }
      before += __popc(ms);
      ties += __popc(mt);
    }
  }
}

template <int G>
int launch_one(cudaLaunchConfig_t& cfg, const SelectParams& p) {
  if (!ensure_smem<select_kernel<G>>(kSmemCap)) return -2;
  return cudaLaunchKernelEx(&cfg, select_kernel<G>, p) == cudaSuccess ? 0 : -2;
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
  while (Q > 1 && (select_smem(Q, p.group, p.max_pages_per_seq) > 100 * 1024 || tiles(Q) < num_sms)) Q /= 2;
  p.queries = Q;
  // CTAs that share a tile's pages: while the grid has room for them and each keeps two page
  // tiles per warp.
  const int ptiles = (p.max_pages_per_seq + 15) / 16;
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
