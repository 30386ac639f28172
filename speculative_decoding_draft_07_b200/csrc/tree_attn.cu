// Tree attention, host side: which kernel takes a call, its workspace and parameters.
#include <algorithm>

#include "attn_sched.cuh"

namespace pct {

// attn_mma.cu: bf16, any page size, head_dim up to 256
int attn_mma_rows(int rows);
int attn_mma_blocks(int d);
cudaError_t launch_attn_mma(const AttnParams& p, int bm, int grid, cudaStream_t s);
// attn_f32.cu: fp32; the same rows a block
int attn_f32_blocks(int d);
cudaError_t launch_attn_f32(const AttnParams& p, int bm, int grid, cudaStream_t s);
// attn_umma.cu
int attn_umma_rows();
bool attn_umma_pages(int page_size);
cudaError_t launch_attn_umma(AttnParams p, int grid, cudaStream_t s);

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

struct AttnPlan {
  bool umma;                    // try the tcgen05 kernel first
  int bm, grid;                 // of the other kernels
  size_t o_po, o_ml, o_meta, o_fail, total;
};
AttnPlan plan(const kv_cache_desc& kv, int batch, int n, int hq) {
  AttnPlan P;
  const int g = hq / kv.heads_kv;
  const long long rows = (long long)n * g;
  // The tcgen05 kernel from 33 rows on (32 requests of 500 to 32768 tokens, 8 heads of
  // 128: 64 rows take 765 us on the warp-level kernel and 440 us on this one, 32 rows
  // 369 us there), where its tiles can hold the rows and the pages.
  P.umma = kv.dtype == PCT_BF16 && rows > 32 && attn_umma_pages(kv.page_size);
  P.bm = attn_mma_rows((int)std::min<long long>(rows, 1 << 20));
  P.grid = num_sms() * (kv.dtype == PCT_BF16 ? attn_mma_blocks(kv.head_dim)
                                             : attn_f32_blocks(kv.head_dim));
  size_t prows = (size_t)P.grid * 2 * P.bm;
  if (P.umma) prows = std::max(prows, (size_t)num_sms() * 2 * attn_umma_rows());
  size_t o = 0;
  P.o_po = o;   o += align_up(prows * kv.head_dim * sizeof(float));
  P.o_ml = o;   o += align_up(prows * sizeof(float2));
  P.o_meta = o; o += align_up((size_t)P.grid * sizeof(int4));
  P.o_fail = o; o += align_up((size_t)P.grid * sizeof(int32_t));
  P.total = o;
  return P;
}

}  // namespace

size_t attn_workspace(const kv_cache_desc& kv, int batch, int n, int hq) {
  return plan(kv, batch, n, hq).total;
}

cudaError_t launch_attn(const AttnArgs& a, void* ws, cudaStream_t s) {
  const AttnPlan P = plan(a.kv, a.batch, a.n, a.hq);
  char* w = static_cast<char*>(ws);
  AttnParams p;
  p.batch = a.batch; p.n = a.n; p.hq = a.hq; p.hkv = a.kv.heads_kv; p.g = a.hq / a.kv.heads_kv;
  p.d = a.kv.head_dim; p.page_size = a.kv.page_size; p.n_pages = a.kv.n_pages;
  p.max_pages = a.kv.max_pages; p.words = (a.n + 31) / 32;
  p.scale_log2 = a.scale * kLog2e;
  p.qs_b = a.qs_b; p.qs_n = a.qs_n; p.qs_h = a.qs_h;
  p.ks_page = a.kv.page_stride; p.ks_slot = a.kv.slot_stride; p.ks_head = a.kv.head_stride;
  p.pg_shift = 0;
  while ((1u << p.pg_shift) < (unsigned)p.page_size) ++p.pg_shift;
  p.pg_mul = (uint32_t)(((1ull << 32) * ((1ull << p.pg_shift) - p.page_size)) / p.page_size + 1);
  p.q = a.q; p.k = a.k; p.v = a.v; p.table = a.table; p.ctx_len = a.ctx_len; p.count = a.count;
  p.mask = a.mask; p.out = a.out; p.lse = a.lse; p.status = a.status;
  p.po = reinterpret_cast<float*>(w + P.o_po);
  p.pml = reinterpret_cast<float2*>(w + P.o_ml);
  p.meta = reinterpret_cast<int4*>(w + P.o_meta);
  p.fail = reinterpret_cast<int32_t*>(w + P.o_fail);
  p.bm = p.half = P.bm;
  p.few = p.many = 1;
  p.per_item = 0;
  // the tcgen05 kernel scales masked (-inf) scores and takes maxima before scaling
  if (P.umma && a.scale > 0.f) {
    const cudaError_t e = launch_attn_umma(p, num_sms(), s);
    if (e != cudaErrorNotSupported) return e;   // strides a tensor map cannot hold: the other kernel
  }
  return a.kv.dtype == PCT_BF16 ? launch_attn_mma(p, P.bm, P.grid, s)
                                : launch_attn_f32(p, P.bm, P.grid, s);
}

}  // namespace pct
