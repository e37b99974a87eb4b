// kvq_internal.h -- parameter blocks shared by the host code and the kernels of libkvq.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/kvq.h"

namespace kvq {

// Dynamic shared memory of a kernel raised to `bytes`: an attribute of the function in the
// current device's context, set once per device (devices 64 and up set it on every launch).
template <auto Kernel>
bool ensure_smem(size_t bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
  if (bit == 0 || (done.load(std::memory_order_acquire) & bit) == 0) {
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) !=
        cudaSuccess)
      return false;
    done.fetch_or(bit, std::memory_order_release);
  }
  return true;
}

// Descriptor validation shared by every entry point that takes a kvq_desc: true when the
// geometry is one the kernels implement; otherwise *why is KVQ_EINVAL (a null descriptor,
// a non-positive size) or KVQ_EUNSUPPORTED (a shape outside the kernels).
bool desc_valid(const kvq_desc* d, int* why);
// Bytes of one token row of a (page, head) block (132 INT4, 144 NVFP4) and of one layer of
// the pool; desc_valid(d) must hold.
size_t desc_row_bytes(const kvq_desc* d);
size_t desc_layer_bytes(const kvq_desc* d);

// Device status bits (same values as KVQ_DEV_* in include/kvq.h).
constexpr int KVQ_DEV_BAD_PAGE_BIT = 1;
constexpr int KVQ_DEV_BAD_POS_BIT = 2;
constexpr int KVQ_DEV_TIMEOUT_BIT = 4;

struct AppendParams {
  uint8_t* pool_layer;            // block(0, 0) of the layer
  const __half* k;                // [T][Hkv][128]
  const __half* v;                // [T][Hkv][128]
  const int32_t* cu_new_tokens;   // [batch+1]
  const int32_t* seq_lens;        // [batch], before the append
  const int32_t* page_table;      // [batch][max_pages_per_seq]
  int32_t* status;                // device status word
  int batch;
  int total_new_tokens;
  int num_kv_heads;
  int num_pages;
  int page_size;
  int max_pages_per_seq;
  float cb;                       // fp32 nearest 1/sqrt(hadamard_block)
  int fp4;                        // 1: NVFP4 rows (E2M1 codes, E4M3 scale per 16 channels)
  int page_shift;                 // log2(page_size)
  // n / num_kv_heads for 0 <= n < 2^31 as umulhi(2n, heads_magic) >> heads_shift
  uint32_t heads_magic;
  int heads_shift;
};

// Tokens per decode tile (one shared-memory ring slot per tile).
constexpr int kTileTokens = 32;
// fp32 words per (partial, query) record in the split scratch: o'[128], m, l, 2 pad.
constexpr int kPartStride = 132;
// Warps per decode CTA; each (unit, CTA) partial slot holds one record per warp.
constexpr int kDecodeWarps = 4;

struct DecodeParams {
  const uint8_t* pool_layer;      // block(0, 0) of the layer
  const __half* q;                // [batch][Hq][128]
  const int32_t* seq_lens;        // [batch], tokens to attend
  const int32_t* page_table;      // [batch][max_pages_per_seq]
  __half* out;                    // [batch][Hq][128]
  float* part;                    // per-(unit, CTA) partials [slots][G][kPartStride]
  int32_t* counters;              // [max_batch * Hkv] arrival counters, zero between calls
  int32_t* status;
  int batch;
  int num_kv_heads;
  int group;                      // G = Hq / Hkv
  int num_pages;
  int page_size;
  int page_shift;                 // log2(page_size)
  int max_pages_per_seq;
  int hadamard_block;
  float q_scale;                  // softmax_scale * log2(e)
  float cb;                       // fp32 nearest 1/sqrt(hadamard_block)
  int total_ctas;                 // C: CTAs in the grid
  // Fused one-token append (null for a plain decode): the new K and V rows [batch][Hkv][128]
  // are rotated, quantised and stored at position seq_lens[b], and the decode runs over
  // seq_lens[b] + 1 tokens (the pool is then written through pool_layer).
  const __half* k_new;
  const __half* v_new;
  int fp4;                        // 1: NVFP4 cache (host-side kernel choice)
};

struct PrefillParams {
  const uint8_t* pool_layer;      // block(0, 0) of the layer
  const __half* q;                // [total_q][Hq][128], chunks concatenated by sequence
  const int32_t* cu_q;            // [batch+1] chunk offsets
  const int32_t* seq_lens;        // [batch] tokens cached, the chunk included
  const int32_t* page_table;      // [batch][max_pages_per_seq]
  __half* out;                    // [total_q][Hq][128]
  int32_t* status;
  int batch;
  int num_kv_heads;
  int group;
  int num_pages;
  int page_size;
  int page_shift;
  int max_pages_per_seq;
  int hadamard_block;
  float q_scale;                  // softmax_scale * log2(e)
  float cb;
  int total_q;                    // rows of q and out
  int fp4;                        // 1: NVFP4 cache
};

// Host-side launchers (return 0 on success, <0 on an unsupported shape or a launch
// error).
int launch_append(const AppendParams& p, int block, int num_sms, cudaStream_t stream);
// Chunked prefill on the 5th-generation tensor cores (INT4 and NVFP4 caches).
int launch_prefill_tc(const PrefillParams& p, int total_q, cudaStream_t stream);

// Append with the position rotation of q and k: k, v and q (null: none) fp16 or bf16, token
// strides in elements.
struct RopeAppendParams {
  uint8_t* pool_layer;
  const void* q;                  // [T] tokens of [Hq][128], or null
  const void* k;                  // [T] tokens of [Hkv][128]
  const void* v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* cu_new_tokens;   // [batch+1]
  const int32_t* seq_lens;        // [batch], before the append
  const int32_t* positions;       // [T] positions of the angles, or null: the cache positions
  const int32_t* page_table;
  const float* inv_freq;          // [rotary_dim / 2]
  __half* q_out;                  // [T][Hq][128]
  int32_t* status;
  double factor;                  // multiplies cosines and sines
  int rotary_dim;
  int interleaved;
  int batch;
  int total_new_tokens;
  int num_kv_heads;
  int group;
  int num_pages;
  int page_size;
  int page_shift;
  int max_pages_per_seq;
  float cb;
  int tile_tokens, tile_heads;    // set by the launcher
};

// Cached rows back in the model's basis.
struct GatherParams {
  const uint8_t* pool_layer;
  const int32_t* cu_rows;         // [batch+1]
  const int32_t* starts;          // [batch] first position of each sequence's range
  const int32_t* page_table;
  void* k_out;                    // [T][Hkv][128] or null
  void* v_out;
  int32_t* status;
  int batch;
  int total_rows;
  int num_kv_heads;
  int num_pages;
  int page_size;
  int page_shift;
  int max_pages_per_seq;
  float cb;
};

// Per-page key bounds.
struct BoundsParams {
  const uint8_t* pool_layer;
  int8_t* codes;                  // [num_pages][Hkv][2][128] of the layer
  float* scale;                   // [num_pages][Hkv] of the layer
  const int32_t* cu_new_tokens;
  const int32_t* seq_lens;        // before the append
  const int32_t* page_table;
  int32_t* status;
  int batch;
  int total_new_tokens;
  int num_kv_heads;
  int num_pages;
  int page_size;
  int page_shift;
  int max_pages_per_seq;
};

// Pages chosen per query and KV head by the bounds' score.
struct SelectParams {
  const int8_t* codes;            // of the layer, as BoundsParams
  const float* scale;
  const __half* q;                // [total_q][Hq][128]
  const int32_t* cu_q;            // [batch+1], or null: one query per sequence
  const int32_t* seq_lens;        // [batch], the queries' own tokens included
  const int32_t* page_table;
  int32_t* blocks;                // [total_q][Hkv][num_blocks]
  int32_t* status;
  int batch;
  int total_q;
  int num_kv_heads;
  int group;
  int num_pages;
  int page_size;
  int page_shift;
  int max_pages_per_seq;
  int hadamard_block;
  float cb;
  int num_blocks, sink, recent;
  int queries;                    // queries of one CTA's tile (set by the launcher)
};

struct SparseParams {
  const int32_t* cu_q;            // [batch+1], or null
  const int32_t* blocks;          // [total_q][Hkv][num_blocks]
  int num_blocks;
  int total_q;
  int num_counters;               // arrival counters of the handle
  long long num_slots;            // partial records of G queries in the scratch
};

// Host-side launchers of the position-rotating append, the read-back, and block-sparse
// attention with its bounds and selection.
int launch_rope_append(RopeAppendParams p, int block, bool fp4, bool bf16, int num_sms, cudaStream_t stream);
int launch_gather(const GatherParams& p, int block, bool fp4, bool bf16, cudaStream_t stream);
int launch_bounds(const BoundsParams& p, bool fp4, cudaStream_t stream);
int launch_select(SelectParams p, int num_sms, cudaStream_t stream);

struct DecodeLaunch {
  int grid;          // CTAs (a multiple of the SM count)
  size_t smem;       // dynamic shared memory per CTA
};
// Shape of the decode pass for a batch capacity (grid sized to fill every SM).
int plan_decode(int group, int page_size, int max_batch, int num_sms, int fp4, DecodeLaunch* out);
int launch_decode(const DecodeParams& p, const DecodeLaunch& L, cudaStream_t stream);
// Attention over chosen pages: p as for a decode (batch sequences), sp the queries and lists.
int launch_sparse(const DecodeParams& p, const SparseParams& sp, int num_sms, cudaStream_t stream);

}  // namespace kvq

struct kvq_cache {
  kvq_desc d;
  uint8_t* pool;
  size_t pool_bytes;
  bool own_pool;
  void* scratch;             // one allocation: status word, unit counters, partials
  int32_t* status;
  int32_t* counters;
  float* part;
  int device;
  int num_sms;
  kvq::DecodeLaunch launch;  // split-pass shape, fixed for the handle
  float cb;
};
