// C ABI of the paged cache and tree attention: argument checks and launches.
// Like the rest of the ABI, nothing here synchronises or allocates.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "internal.h"

using namespace pct;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// stride of rows that are read and written 16 bytes at a time
bool stride_ok(int64_t s, int per) { return s >= 0 && s % per == 0; }

int check_cache(const kv_cache_desc* d) {
  if (!d) return PCT_EINVAL;
  if (d->dtype != PCT_F32 && d->dtype != PCT_BF16) return PCT_EINVAL;
  if (d->n_pages < 1 || d->page_size < 1 || d->page_size > 65536 || d->max_pages < 1)
    return PCT_EINVAL;
  if ((int64_t)d->max_pages * d->page_size > (1ll << 30)) return PCT_EINVAL;
  if (d->heads_kv < 1 || d->heads_kv > 1024) return PCT_EINVAL;
  if (d->head_dim < 8 || d->head_dim > 256 || d->head_dim % 8 != 0) return PCT_EINVAL;
  const int per = d->dtype == PCT_BF16 ? 8 : 4;
  if (!stride_ok(d->page_stride, per) || !stride_ok(d->slot_stride, per) ||
      !stride_ok(d->head_stride, per))
    return PCT_EINVAL;
  return PCT_OK;
}
// For the calls that write: rows of a cache apart from each other. (An axis of stride 0, as an
// expanded view has it, would be written by several blocks at once.)
bool rows_apart(int64_t n, int64_t stride, int d) { return n == 1 || stride >= d; }
bool writable(const kv_cache_desc& d) {
  return rows_apart(d.n_pages, d.page_stride, d.head_dim) &&
         rows_apart(d.page_size, d.slot_stride, d.head_dim) &&
         rows_apart(d.heads_kv, d.head_stride, d.head_dim);
}
bool batch_ok(int32_t batch) { return batch >= 1 && batch <= 65535; }
bool table_ok(int32_t page_size, int32_t max_pages, int32_t n_pages) {
  return page_size >= 1 && page_size <= 65536 && max_pages >= 1 && n_pages >= 1 &&
         (int64_t)max_pages * page_size <= (1ll << 30);
}
int check_attn(const kv_cache_desc* d, int32_t batch, int32_t n, int32_t hq) {
  const int st = check_cache(d);
  if (st != PCT_OK) return st;
  if (!batch_ok(batch) || n < 1 || n > 65536) return PCT_EINVAL;
  if (hq < 1 || hq % d->heads_kv != 0 || hq / d->heads_kv > 64) return PCT_EINVAL;
  return PCT_OK;
}

// A call's dense array (null: not given). Blocks read lengths, counts, tables and paths at
// different times and rely on reading the same values, so an output that overlaps one of
// them would take indices and barriers out of step.
struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && a.bytes && b.bytes && (x < y ? y - x < a.bytes : x - y < b.bytes);
}
// outputs apart from each other and from the inputs
bool disjoint(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* a = outs.begin(); a != outs.end(); ++a) {
    for (const Span* b = a + 1; b != outs.end(); ++b)
      if (overlap(*a, *b)) return false;
    for (const Span& b : ins)
      if (overlap(*a, b)) return false;
  }
  return true;
}

#define PCT_CU(x)                             \
  do {                                        \
    if ((x) != cudaSuccess) return PCT_ECUDA; \
  } while (0)

}  // namespace

extern "C" {

int32_t kv_pages_resize(int32_t batch, int32_t page_size, int32_t max_pages, int32_t n_pages,
                        const int64_t* ctx_len, const int32_t* count, int32_t* block_table,
                        int32_t* held, int32_t* free_pages, int32_t* free_count,
                        int32_t* dev_status, void* cuda_stream) {
  if (!batch_ok(batch) || !table_ok(page_size, max_pages, n_pages)) return PCT_EINVAL;
  if (!ctx_len || !block_table || !held || !free_pages || !free_count || !dev_status)
    return PCT_EINVAL;
  const size_t nb = batch;
  if (!disjoint({{block_table, nb * max_pages * 4}, {held, nb * 4}, {free_pages, (size_t)n_pages * 4},
                 {free_count, 4}, {dev_status, nb * 4}},
                {{ctx_len, nb * 8}, {count, nb * 4}}))
    return PCT_EINVAL;
  if (!device_ok()) return PCT_EDEVICE;
  PCT_CU(launch_kv_pages_resize(batch, page_size, max_pages, n_pages, ctx_len, count, block_table,
                                held, free_pages, free_count, dev_status,
                                static_cast<cudaStream_t>(cuda_stream)));
  return PCT_OK;
}

int32_t kv_tree_slots(int32_t batch, int32_t n_stride, int32_t page_size, int32_t max_pages,
                      int32_t n_pages, const int64_t* ctx_len, const int32_t* count,
                      const int32_t* depth, const int32_t* block_table, int64_t* slot,
                      int64_t* pos, int32_t* dev_status, void* cuda_stream) {
  if (!batch_ok(batch) || n_stride < 1 || n_stride > (1 << 20) ||
      !table_ok(page_size, max_pages, n_pages))
    return PCT_EINVAL;
  if (!ctx_len || !count || !block_table || !slot || !pos || !dev_status) return PCT_EINVAL;
  const size_t nb = batch, rows = nb * n_stride;
  if (!disjoint({{slot, rows * 8}, {pos, rows * 8}, {dev_status, nb * 4}},
                {{ctx_len, nb * 8}, {count, nb * 4}, {depth, rows * 4}, {block_table, nb * max_pages * 4}}))
    return PCT_EINVAL;
  if (!device_ok()) return PCT_EDEVICE;
  PCT_CU(launch_kv_tree_slots(batch, n_stride, page_size, max_pages, n_pages, ctx_len, count,
                              depth, block_table, slot, pos, dev_status,
                              static_cast<cudaStream_t>(cuda_stream)));
  return PCT_OK;
}

int32_t kv_append(const kv_cache_desc* desc, int32_t batch, int32_t n_stride, const void* k_new,
                  const void* v_new, const int64_t* new_stride, const int64_t* slot,
                  void* k_cache, void* v_cache, int32_t* dev_status, void* cuda_stream) {
  const int st = check_cache(desc);
  if (st != PCT_OK) return st;
  if (!batch_ok(batch) || n_stride < 1 || n_stride > (1 << 20) || !writable(*desc)) return PCT_EINVAL;
  if (!k_new || !v_new || !new_stride || !slot || !k_cache || !v_cache || !dev_status)
    return PCT_EINVAL;
  const int per = desc->dtype == PCT_BF16 ? 8 : 4;
  for (int i = 0; i < 3; ++i)
    if (!stride_ok(new_stride[i], per)) return PCT_EINVAL;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return PCT_EINVAL;
  if (overlap({dev_status, (size_t)batch * 4}, {slot, (size_t)batch * n_stride * 8})) return PCT_EINVAL;
  if (!device_ok()) return PCT_EDEVICE;
  PCT_CU(launch_kv_append(*desc, batch, n_stride, k_new, v_new, new_stride, slot, k_cache, v_cache,
                          dev_status, static_cast<cudaStream_t>(cuda_stream)));
  return PCT_OK;
}

size_t tree_attention_workspace(const kv_cache_desc* desc, int32_t batch, int32_t n_stride,
                                int32_t heads_q) {
  if (check_attn(desc, batch, n_stride, heads_q) != PCT_OK) return 0;
  return attn_workspace(*desc, batch, n_stride, heads_q);
}

int32_t tree_attention(const kv_cache_desc* desc, int32_t batch, int32_t n_stride,
                       int32_t heads_q, float scale, const void* q, const int64_t* q_stride,
                       const void* k_cache, const void* v_cache, const int32_t* block_table,
                       const int64_t* ctx_len, const int32_t* count, const uint32_t* mask,
                       void* out, float* lse, int32_t* dev_status, void* workspace,
                       size_t ws_bytes, void* cuda_stream) {
  const int st = check_attn(desc, batch, n_stride, heads_q);
  if (st != PCT_OK) return st;
  if (!q || !q_stride || !k_cache || !v_cache || !block_table || !ctx_len || !out || !dev_status)
    return PCT_EINVAL;
  if (!std::isfinite(scale * 1.4426950f)) return PCT_EINVAL;   // the kernels' base-2 scale
  const int per = desc->dtype == PCT_BF16 ? 8 : 4;
  for (int i = 0; i < 3; ++i)
    if (!stride_ok(q_stride[i], per)) return PCT_EINVAL;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
    return PCT_EINVAL;
  const size_t nb = batch, rows = nb * n_stride;
  const size_t need = attn_workspace(*desc, batch, n_stride, heads_q);
  if (!disjoint({{out, rows * heads_q * desc->head_dim * (desc->dtype == PCT_BF16 ? 2 : 4)},
                 {lse, rows * heads_q * 4}, {dev_status, nb * 4}, {workspace, std::min(need, ws_bytes)}},
                {{block_table, nb * desc->max_pages * 4}, {ctx_len, nb * 8}, {count, nb * 4},
                 {mask, rows * ((n_stride + 31) / 32) * 4}}))
    return PCT_EINVAL;
  if (!device_ok()) return PCT_EDEVICE;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < need) return PCT_EWORKSPACE;
  AttnArgs a;
  a.kv = *desc;
  a.batch = batch; a.n = n_stride; a.hq = heads_q; a.scale = scale;
  a.q = q; a.qs_b = q_stride[0]; a.qs_n = q_stride[1]; a.qs_h = q_stride[2];
  a.k = k_cache; a.v = v_cache; a.table = block_table; a.ctx_len = ctx_len; a.count = count;
  a.mask = mask; a.out = out; a.lse = lse; a.status = dev_status;
  PCT_CU(launch_attn(a, workspace, static_cast<cudaStream_t>(cuda_stream)));
  return PCT_OK;
}

int32_t kv_commit(const kv_cache_desc* desc, int32_t batch, int32_t layers, int64_t layer_stride,
                  int32_t max_depth, void* k_cache, void* v_cache, const int32_t* block_table,
                  const int64_t* ctx_len, const int32_t* count, const int32_t* accept_len,
                  const int32_t* accept_path, int64_t* new_len, int32_t* dev_status,
                  void* cuda_stream) {
  const int st = check_cache(desc);
  if (st != PCT_OK) return st;
  if (!batch_ok(batch) || layers < 1 || layers > 65535 || max_depth < 1 || max_depth > 4096)
    return PCT_EINVAL;
  if (!k_cache || !v_cache || !block_table || !ctx_len || !count || !accept_len || !accept_path ||
      !new_len || !dev_status)
    return PCT_EINVAL;
  if (!stride_ok(layer_stride, desc->dtype == PCT_BF16 ? 8 : 4)) return PCT_EINVAL;
  if (!writable(*desc) || !rows_apart(layers, layer_stride, desc->head_dim)) return PCT_EINVAL;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return PCT_EINVAL;
  const size_t nb = batch;
  if (!disjoint({{new_len, nb * 8}, {dev_status, nb * 4}},
                {{block_table, nb * desc->max_pages * 4}, {ctx_len, nb * 8}, {count, nb * 4},
                 {accept_len, nb * 4}, {accept_path, nb * max_depth * 4}}))
    return PCT_EINVAL;
  if (!device_ok()) return PCT_EDEVICE;
  PCT_CU(launch_kv_commit(*desc, batch, layers, layer_stride, max_depth, k_cache, v_cache,
                          block_table, ctx_len, count, accept_len, accept_path, new_len,
                          dev_status, static_cast<cudaStream_t>(cuda_stream)));
  return PCT_OK;
}

}  // extern "C"
