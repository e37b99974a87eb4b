// kvq_ops.cu -- host side of the calls around the cache: the append with the position rotation,
// the read-back of rows, and block-sparse attention with its page bounds and page choice.
// Argument checks (all before any launch), parameter blocks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/kvq.h"
#include "kvq_internal.h"

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The checks that every call shares: the handle, its device, the layer and the batch.
int check_call(const kvq_cache* c, int32_t layer, int32_t batch, int32_t total) {
  if (!c) return KVQ_EINVAL;
  if (layer < 0 || layer >= c->d.num_layers) return KVQ_EINVAL;
  if (batch < 0 || batch > c->d.max_batch || total < 0) return KVQ_EINVAL;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVQ_ECUDA;
  if (dev != c->device) return KVQ_EINVAL;  // a launch here would read another device's memory
  return KVQ_OK;
}

uint8_t* layer_of(const kvq_cache* c, int32_t layer) {
  return c->pool + static_cast<size_t>(layer) * kvq::desc_layer_bytes(&c->d);
}

int shift_of(const kvq_cache* c) { return __builtin_ctz(static_cast<unsigned>(c->d.page_size)); }

bool fp4_of(const kvq_cache* c) { return c->d.kv_format == KVQ_FORMAT_NVFP4; }

int group_of(const kvq_cache* c) { return c->d.num_q_heads / c->d.num_kv_heads; }

int status_of(int rc) { return rc == 0 ? KVQ_OK : rc == -1 ? KVQ_EUNSUPPORTED : KVQ_ECUDA; }

}  // namespace

extern "C" {

int kvq_rope_quant_append(kvq_cache* c, int32_t layer, int32_t dtype, const void* q, int64_t q_stride,
                          const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const int32_t* cu_new_tokens, const int32_t* seq_lens, const int32_t* positions,
                          const int32_t* page_table, int32_t batch, int32_t total_new_tokens,
                          const float* inv_freq, int32_t rotary_dim, int32_t interleaved, double factor,
                          void* q_out, void* stream) {
  const int rc = check_call(c, layer, batch, total_new_tokens);
  if (rc != KVQ_OK) return rc;
  if (dtype != KVQ_DTYPE_FP16 && dtype != KVQ_DTYPE_BF16) return KVQ_EINVAL;
  if (rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16) return KVQ_EUNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return KVQ_EINVAL;
  if (!isfinite(factor)) return KVQ_EINVAL;
  if (total_new_tokens == 0) return KVQ_OK;
  if (batch == 0) return KVQ_EINVAL;
  if (!k || !v || !cu_new_tokens || !seq_lens || !page_table || !inv_freq) return KVQ_EINVAL;
  if ((q == nullptr) != (q_out == nullptr)) return KVQ_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16)) return KVQ_EINVAL;
  // Token strides: whole 16-byte units, at least a token's rows (0 for a single token).
  const int64_t kv_row = static_cast<int64_t>(c->d.num_kv_heads) * 128;
  const int64_t q_row = static_cast<int64_t>(c->d.num_q_heads) * 128;
  const bool one = total_new_tokens == 1;
  if (k_stride % 8 || v_stride % 8 || (!one && (k_stride < kv_row || v_stride < kv_row))) return KVQ_EINVAL;
  if (q && (q_stride % 8 || (!one && q_stride < q_row))) return KVQ_EINVAL;
  kvq::RopeAppendParams p = {};
  p.pool_layer = layer_of(c, layer);
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.cu_new_tokens = cu_new_tokens;
  p.seq_lens = seq_lens;
  p.positions = positions;
  p.page_table = page_table;
  p.inv_freq = inv_freq;
  p.q_out = static_cast<__half*>(q_out);
  p.status = c->status;
  p.factor = factor;
  p.rotary_dim = rotary_dim;
  p.interleaved = interleaved;
  p.batch = batch;
  p.total_new_tokens = total_new_tokens;
  p.num_kv_heads = c->d.num_kv_heads;
  p.group = group_of(c);
  p.num_pages = c->d.num_pages;
  p.page_size = c->d.page_size;
  p.page_shift = shift_of(c);
  p.max_pages_per_seq = c->d.max_pages_per_seq;
  p.cb = c->cb;
  return status_of(kvq::launch_rope_append(p, c->d.hadamard_block, fp4_of(c), dtype == KVQ_DTYPE_BF16, c->num_sms,
                                           static_cast<cudaStream_t>(stream)));
}

int kvq_gather_rows(kvq_cache* c, int32_t layer, const int32_t* cu_rows, const int32_t* starts,
                    const int32_t* page_table, int32_t batch, int32_t total_rows, int32_t dtype, void* k_out,
                    void* v_out, void* stream) {
  const int rc = check_call(c, layer, batch, total_rows);
  if (rc != KVQ_OK) return rc;
  if (dtype != KVQ_DTYPE_FP16 && dtype != KVQ_DTYPE_BF16) return KVQ_EINVAL;
  if (total_rows == 0) return KVQ_OK;
  if (batch == 0 || !cu_rows || !starts || !page_table || (!k_out && !v_out)) return KVQ_EINVAL;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return KVQ_EINVAL;  // bulk copies
  kvq::GatherParams p = {};
  p.pool_layer = layer_of(c, layer);
  p.cu_rows = cu_rows;
  p.starts = starts;
  p.page_table = page_table;
  p.k_out = k_out;
  p.v_out = v_out;
  p.status = c->status;
  p.batch = batch;
  p.total_rows = total_rows;
  p.num_kv_heads = c->d.num_kv_heads;
  p.num_pages = c->d.num_pages;
  p.page_size = c->d.page_size;
  p.page_shift = shift_of(c);
  p.max_pages_per_seq = c->d.max_pages_per_seq;
  p.cb = c->cb;
  return status_of(kvq::launch_gather(p, c->d.hadamard_block, fp4_of(c), dtype == KVQ_DTYPE_BF16,
                                      static_cast<cudaStream_t>(stream)));
}

int kvq_update_block_bounds(kvq_cache* c, int32_t layer, void* codes, float* scale, const int32_t* cu_new_tokens,
                            const int32_t* seq_lens, const int32_t* page_table, int32_t batch,
                            int32_t total_new_tokens, void* stream) {
  const int rc = check_call(c, layer, batch, total_new_tokens);
  if (rc != KVQ_OK) return rc;
  if (total_new_tokens == 0) return KVQ_OK;
  if (batch == 0 || !codes || !scale || !cu_new_tokens || !seq_lens || !page_table) return KVQ_EINVAL;
  if (!aligned(codes, 32) || !aligned(scale, 4)) return KVQ_EINVAL;
  const size_t rows = static_cast<size_t>(layer) * c->d.num_pages * c->d.num_kv_heads;
  kvq::BoundsParams p = {};
  p.pool_layer = layer_of(c, layer);
  p.codes = static_cast<int8_t*>(codes) + rows * 256;
  p.scale = scale + rows;
  p.cu_new_tokens = cu_new_tokens;
  p.seq_lens = seq_lens;
  p.page_table = page_table;
  p.status = c->status;
  p.batch = batch;
  p.total_new_tokens = total_new_tokens;
  p.num_kv_heads = c->d.num_kv_heads;
  p.num_pages = c->d.num_pages;
  p.page_size = c->d.page_size;
  p.page_shift = shift_of(c);
  p.max_pages_per_seq = c->d.max_pages_per_seq;
  return status_of(kvq::launch_bounds(p, fp4_of(c), static_cast<cudaStream_t>(stream)));
}

int kvq_select_blocks(kvq_cache* c, int32_t layer, const void* codes, const float* scale, const void* q,
                      const int32_t* cu_q, const int32_t* seq_lens, const int32_t* page_table, int32_t batch,
                      int32_t total_q, int32_t num_blocks, int32_t sink, int32_t recent, int32_t* blocks,
                      void* stream) {
  const int rc = check_call(c, layer, batch, total_q);
  if (rc != KVQ_OK) return rc;
  if (num_blocks < 1 || sink < 0 || recent < 0 || sink > num_blocks || recent > num_blocks - sink) return KVQ_EINVAL;
  if (!cu_q && total_q != batch) return KVQ_EINVAL;
  if (batch == 0 || total_q == 0) return KVQ_OK;
  if (!codes || !scale || !q || !seq_lens || !page_table || !blocks) return KVQ_EINVAL;
  if (!aligned(codes, 32) || !aligned(scale, 4) || !aligned(q, 16)) return KVQ_EINVAL;  // 256-bit loads
  const size_t rows = static_cast<size_t>(layer) * c->d.num_pages * c->d.num_kv_heads;
  kvq::SelectParams p = {};
  p.codes = static_cast<const int8_t*>(codes) + rows * 256;
  p.scale = scale + rows;
  p.q = static_cast<const __half*>(q);
  p.cu_q = cu_q;
  p.seq_lens = seq_lens;
  p.page_table = page_table;
  p.blocks = blocks;
  p.status = c->status;
  p.batch = batch;
  p.total_q = total_q;
  p.num_kv_heads = c->d.num_kv_heads;
  p.group = group_of(c);
  p.num_pages = c->d.num_pages;
  p.page_size = c->d.page_size;
  p.page_shift = shift_of(c);
  p.max_pages_per_seq = c->d.max_pages_per_seq;
  p.hadamard_block = c->d.hadamard_block;
  p.cb = c->cb;
  p.num_blocks = num_blocks;
  p.sink = sink;
  p.recent = recent;
  return status_of(kvq::launch_select(p, c->num_sms, static_cast<cudaStream_t>(stream)));
}

int kvq_sparse_attention(kvq_cache* c, int32_t layer, const void* q, const int32_t* cu_q, const int32_t* seq_lens,
                         const int32_t* page_table, const int32_t* blocks, int32_t num_blocks, int32_t batch,
                         int32_t total_q, float softmax_scale, void* out, void* stream) {
  const int rc = check_call(c, layer, batch, total_q);
  if (rc != KVQ_OK) return rc;
  if (!(softmax_scale >= 0.0f) || isinf(softmax_scale)) return KVQ_EINVAL;
  if (num_blocks < 1) return KVQ_EINVAL;
  if (static_cast<long long>(num_blocks) * c->d.page_size > (1LL << 30)) return KVQ_EUNSUPPORTED;
  if (!cu_q && total_q != batch) return KVQ_EINVAL;
  if (batch == 0 || total_q == 0) return KVQ_OK;
  if (!q || !seq_lens || !page_table || !blocks || !out) return KVQ_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16)) return KVQ_EINVAL;
  kvq::DecodeParams p = {};
  p.pool_layer = layer_of(c, layer);
  p.q = static_cast<const __half*>(q);
  p.seq_lens = seq_lens;
  p.page_table = page_table;
  p.out = static_cast<__half*>(out);
  p.part = c->part;
  p.counters = c->counters;
  p.status = c->status;
  p.batch = batch;
  p.num_kv_heads = c->d.num_kv_heads;
  p.group = group_of(c);
  p.num_pages = c->d.num_pages;
  p.page_size = c->d.page_size;
  p.page_shift = shift_of(c);
  p.max_pages_per_seq = c->d.max_pages_per_seq;
  p.hadamard_block = c->d.hadamard_block;
  const double sm = softmax_scale == 0.0f ? 1.0 / sqrt(static_cast<double>(c->d.head_dim))
                                          : static_cast<double>(softmax_scale);
  p.q_scale = static_cast<float>(sm * 1.4426950408889634);  // log2(e)
  p.cb = c->cb;
  p.fp4 = fp4_of(c);
  kvq::SparseParams sp = {};
  sp.cu_q = cu_q;
  sp.blocks = blocks;
  sp.num_blocks = num_blocks;
  sp.total_q = total_q;
  const long long units = static_cast<long long>(c->d.max_batch) * c->d.num_kv_heads + c->launch.grid;
  sp.num_counters = units < 0x7fffffffLL ? static_cast<int>(units) : 0x7fffffff;
  sp.num_slots = units * kvq::kDecodeWarps;
  return status_of(kvq::launch_sparse(p, sp, c->num_sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
