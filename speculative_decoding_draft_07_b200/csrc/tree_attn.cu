// Tree attention: the host side that picks a kernel, and the kernel for fp32
// caches, on the FP32 pipes.
//
// One pass over the keys with the running maximum and sum of the softmax. A
// block of 128 threads holds BM = 8 * RPT rows of Q in shared memory and steps
// through key tiles of BK = 32 tokens, which arrive by 16-byte asynchronous copies
// two or three tiles ahead (their places worked out one tile before that, a thread a
// token): scores as 8 x 16 thread cells of RPT x 2, the softmax by the 16 threads of
// a row group, and the weighted sum of V as cells of RPT rows x head_dim / 16 columns
// in registers. fp32 products have no tensor path of their own precision, so the FMA
// rate bounds it from about ten rows on, the cache's bytes below.
#include <algorithm>

#include "attn_sched.cuh"

namespace pct {

// attn_mma.cu
int attn_mma_rows(int rows);
int attn_mma_blocks(int d);
cudaError_t launch_attn_mma(const AttnParams& p, int bm, int grid, cudaStream_t s);
// attn_umma.cu
int attn_umma_rows();
bool attn_umma_pages(int page_size);
cudaError_t launch_attn_umma(AttnParams p, int grid, cudaStream_t s);

namespace {

constexpr int kSimtThreads = 128;
constexpr int kSimtBK = 32;

__device__ __forceinline__ void cp16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
template <int DC> struct SimtShape {
  static constexpr int STAGES = DC == 4 ? 3 : 2;
  static constexpr int BLOCKS = DC == 4 ? 3 : DC == 8 ? 2 : 1;   // an SM (shared memory)
};

// DC: columns of head_dim a thread accumulates (head_dim <= 16 * DC).
template <int RPT, int DC>
__global__ void __launch_bounds__(kSimtThreads, SimtShape<DC>::BLOCKS)
attn_simt_kernel(AttnParams p) {
  constexpr int BM = 8 * RPT, BK = kSimtBK, NT = kSimtThreads, STAGES = SimtShape<DC>::STAGES;
  extern __shared__ __align__(16) float sm[];
  __shared__ Share share;
  __shared__ long long sums[NT / 32];
  __shared__ uint32_t seen[BM];            // visible keys of the tile, one bit a key
  __shared__ long long where[4][BK];       // places of a tile's tokens, -1 for none
  __shared__ uint32_t gone[4];             // keys of the tile whose page is bad
  const int dp = p.d + 4;                  // row stride: 16-byte phases of 8 rows differ
  float* Qs = sm;                          // [BM][dp]
  float* ring = Qs + BM * dp;              // [STAGES][K, V][BK][dp]
  float* Ps = ring + STAGES * 2 * BK * dp; // [BK][BM]
  const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15;
  if (tid < 4) gone[tid] = 0;
  pdl_wait();
  pdl_trigger();
  sched_begin<BK, NT>(p, &share, sums);
  int4 begun = make_int4(-1, 0, 0, 0);

  Walk<BK> w;
  w.begin(share);
  while (w.next(p, share, &begun)) {
    const Req r = w.r;
    const int b = w.b, h = w.h, t0 = w.t0, t1 = w.t1, klen = w.klen, rows = w.rows;
    const int row0 = (w.mt - 1) * BM, v4 = p.d / 4;
    const int32_t* table = p.table + (long long)b * p.max_pages;
    const float* kb = static_cast<const float*>(p.k) + h * p.ks_head;
    const float* vb = static_cast<const float*>(p.v) + h * p.ks_head;
    auto find_tile = [&](int t) {
      if (tid >= BK) return;
      const int tok = t * BK + tid;
      long long off = -1;
      if (tok < klen) {
        const uint32_t col = page_of(p, tok);
        const int page = __ldg(table + col);
        if (page >= 0 && page < p.n_pages)
          off = page * p.ks_page + (tok - (int)col * p.page_size) * p.ks_slot;
        else
          atomicOr(&gone[t & 3], 1u << tid);
      }
      where[t & 3][tid] = off;
    };
    auto load_tile = [&](int t) {
      float* kd = ring + (t - t0) % STAGES * 2 * BK * dp;
      for (int i = tid; i < BK * v4; i += NT) {
        const int kk = i / v4, c = (i - kk * v4) * 4;
        const long long at = where[t & 3][kk];
        const long long off = at >= 0 ? at + c : 0;
        cp16(kd + kk * dp + c, kb + off, at >= 0);
        cp16(kd + (BK + kk) * dp + c, vb + off, at >= 0);
      }
    };
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
      if (t0 + i < t1) find_tile(t0 + i);
    for (int i = tid; i < BM * v4; i += NT) {
      const int rr = i / v4, c = (i - rr * v4) * 4;
      const float* src = static_cast<const float*>(p.q);
      if (rr < rows) {
        const int row = row0 + rr, node = row / p.g, qh = h * p.g + (row - node * p.g);
        src += b * p.qs_b + node * p.qs_n + qh * p.qs_h + c;
      }
      cp16(Qs + rr * dp + c, src, rr < rows);          // in the first tile's group
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      if (t0 + i < t1) load_tile(t0 + i);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    float m[RPT], l[RPT];
    float2 acc[RPT][DC / 2];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      m[i] = neg_inf();
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < DC / 2; ++j) acc[i][j] = make_float2(0.f, 0.f);
    }
    for (int t = t0; t < t1; ++t) {
      const float* Ks = ring + (t - t0) % STAGES * 2 * BK * dp;
      const float* Vs = Ks + BK * dp;
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
      if (tid < BM) {
        uint32_t bits = 0;
        if (tid < rows) {
          const int node = (row0 + tid) / p.g;
          bits = seen32(p, p.mask ? p.mask + ((long long)b * p.n + node) * p.words : nullptr, node,
                        t * BK - (int)r.ctx);
        }
        seen[tid] = bits;
      }
      __syncthreads();
      if (t + STAGES - 1 < t1) load_tile(t + STAGES - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (t + STAGES < t1) find_tile(t + STAGES);
      const uint32_t lost = gone[t & 3];
      // packed pairs: even and odd products of a score apart, two columns of V together
      float2 s2[RPT][2];
#pragma unroll
      for (int i = 0; i < RPT; ++i) s2[i][0] = s2[i][1] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < p.d; c += 4) {
        const float4 ka = *reinterpret_cast<const float4*>(Ks + cg * dp + c);
        const float4 kc = *reinterpret_cast<const float4*>(Ks + (cg + 16) * dp + c);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(Qs + (rg * RPT + i) * dp + c);
          const float2 lo = make_float2(x.x, x.y), hi = make_float2(x.z, x.w);
          s2[i][0] = f2_fma(hi, make_float2(ka.z, ka.w), f2_fma(lo, make_float2(ka.x, ka.y), s2[i][0]));
          s2[i][1] = f2_fma(hi, make_float2(kc.z, kc.w), f2_fma(lo, make_float2(kc.x, kc.y), s2[i][1]));
        }
      }
      float s[RPT][2];
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        s[i][0] = s2[i][0].x + s2[i][0].y;
        s[i][1] = s2[i][1].x + s2[i][1].y;
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const uint32_t bits = seen[rg * RPT + i] & ~lost;
        s[i][0] = (bits >> cg) & 1u ? s[i][0] * p.scale_log2 : neg_inf();
        s[i][1] = (bits >> (cg + 16)) & 1u ? s[i][1] * p.scale_log2 : neg_inf();
        float mx = fmaxf(s[i][0], s[i][1]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[i], mx);
        const float ref = mn == neg_inf() ? 0.f : mn;
        const float f = ex2(m[i] - ref);
        const float e0 = ex2(s[i][0] - ref), e1 = ex2(s[i][1] - ref);
        float sum = e0 + e1;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = l[i] * f + sum;
        m[i] = mn;
#pragma unroll
        for (int j = 0; j < DC / 2; ++j) {
          acc[i][j].x *= f;
          acc[i][j].y *= f;
        }
        Ps[cg * BM + rg * RPT + i] = e0;
        Ps[(cg + 16) * BM + rg * RPT + i] = e1;
      }
      __syncthreads();
      if (lost && tid == 0) gone[t & 3] = 0;           // for the ring entry's next tile
#pragma unroll 8
      for (int kk = 0; kk < BK; ++kk) {
        float pr[RPT];
        if constexpr (RPT == 4) {
          const float4 x = *reinterpret_cast<const float4*>(Ps + kk * BM + rg * 4);
          pr[0] = x.x; pr[1] = x.y; pr[2] = x.z; pr[3] = x.w;
        } else if constexpr (RPT == 2) {
          const float2 x = *reinterpret_cast<const float2*>(Ps + kk * BM + rg * 2);
          pr[0] = x.x; pr[1] = x.y;
        } else {
          pr[0] = Ps[kk * BM + rg];
        }
#pragma unroll
        for (int q = 0; q < DC / 4; ++q) {
          const int c = q * 64 + cg * 4;
          if (c < p.d) {
            const float4 v = *reinterpret_cast<const float4*>(Vs + kk * dp + c);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
              const float2 w2 = make_float2(pr[i], pr[i]);
              acc[i][q * 2] = f2_fma(w2, make_float2(v.x, v.y), acc[i][q * 2]);
              acc[i][q * 2 + 1] = f2_fma(w2, make_float2(v.z, v.w), acc[i][q * 2 + 1]);
            }
          }
        }
      }
    }
    const bool whole = w.whole;
    const int slot = w.pslot;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int rr = rg * RPT + i;
      if (rr >= rows) continue;
      if (whole) {
        const int row = row0 + rr, node = row / p.g, qh = h * p.g + (row - node * p.g);
        const long long o = ((long long)b * p.n + node) * p.hq + qh;
        const float inv = inverse(l[i]);
#pragma unroll
        for (int q = 0; q < DC / 4; ++q) {
          const int c = q * 64 + cg * 4;
          if (c < p.d)
            store_out(static_cast<float*>(p.out) + o * p.d + c,
                      make_float4(acc[i][q * 2].x * inv, acc[i][q * 2].y * inv,
                                  acc[i][q * 2 + 1].x * inv, acc[i][q * 2 + 1].y * inv));
        }
        if (p.lse && cg == 0)
          p.lse[o] = lse_of(m[i], l[i]);
      } else {
        const long long at = ((long long)blockIdx.x * 2 + slot) * BM + rr;
#pragma unroll
        for (int q = 0; q < DC / 4; ++q) {
          const int c = q * 64 + cg * 4;
          if (c < p.d)
            *reinterpret_cast<float4*>(p.po + at * p.d + c) = make_float4(
                acc[i][q * 2].x, acc[i][q * 2].y, acc[i][q * 2 + 1].x, acc[i][q * 2 + 1].y);
        }
        if (cg == 0) p.pml[at] = make_float2(m[i], l[i]);
      }
    }
  }
  if (tid == 0) p.meta[blockIdx.x] = begun;
  attn_tail<float>(p);
}

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

struct AttnPlan {
  bool umma;                    // try the tcgen05 kernel first
  int rpt, bm, grid;            // of the other kernels
  size_t o_po, o_ml, o_meta, o_fail, total;
};
AttnPlan plan(const kv_cache_desc& kv, int batch, int n, int hq) {
  AttnPlan P;
  const int g = hq / kv.heads_kv;
  const long long rows = (long long)n * g;
  // The tcgen05 kernel from 33 rows on (32 requests of 500 to 32768 tokens, 8 heads of
  // 128: 64 rows take 765 us on the warp-level kernel and 440 us on this one, 32 rows
  // 369 us there), where its tiles can hold the rows and the pages.
  P.umma = kv.dtype == PCT_BF16 && rows > 32 && kv.head_dim <= 128 && attn_umma_pages(kv.page_size);
  if (kv.dtype == PCT_BF16) {
    P.rpt = 0;
    P.bm = attn_mma_rows((int)std::min<long long>(rows, 1 << 20));
    P.grid = num_sms() * attn_mma_blocks(kv.head_dim);
  } else {
    P.rpt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    P.bm = 8 * P.rpt;
    P.grid = num_sms() * (kv.head_dim <= 64 ? SimtShape<4>::BLOCKS
                          : kv.head_dim <= 128 ? SimtShape<8>::BLOCKS : SimtShape<16>::BLOCKS);
  }
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

template <int RPT, int DC>
cudaError_t run_simt(const AttnParams& p, const AttnPlan& P, cudaStream_t s) {
  constexpr int BM = 8 * RPT;
  const size_t smem = ((size_t)(BM + SimtShape<DC>::STAGES * 2 * kSimtBK) * (p.d + 4) +
                       kSimtBK * BM) * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<RPT, DC>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  {
    TraceScope t(s, "attn_simt");
    e = launch_pdl(attn_simt_kernel<RPT, DC>, dim3(P.grid), dim3(kSimtThreads), smem, s, 1, p);
  }
  if (e != cudaSuccess) return e;
  TraceScope t(s, "attn_join");
  return launch_pdl(attn_join_kernel<float, BM, DC == 16>, dim3(P.grid, (BM + 3) / 4), dim3(128), 0, s, 1, p);
}
template <int RPT>
cudaError_t run_simt_d(const AttnParams& p, const AttnPlan& P, cudaStream_t s) {
  if (p.d <= 64) return run_simt<RPT, 4>(p, P, s);
  if (p.d <= 128) return run_simt<RPT, 8>(p, P, s);
  return run_simt<RPT, 16>(p, P, s);
}
cudaError_t run_simt_r(const AttnParams& p, const AttnPlan& P, cudaStream_t s) {
  if (P.rpt == 1) return run_simt_d<1>(p, P, s);
  if (P.rpt == 2) return run_simt_d<2>(p, P, s);
  return run_simt_d<4>(p, P, s);
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
  p.fail = nullptr;
  p.bm = p.half = P.bm;
  p.few = p.many = 1;
  p.per_item = 0;
  // the tcgen05 kernel scales masked (-inf) scores and takes maxima before scaling
  if (P.umma && a.scale > 0.f) {
    AttnParams up = p;
    up.fail = reinterpret_cast<int32_t*>(w + P.o_fail);
    const cudaError_t e = launch_attn_umma(up, num_sms(), s);
    if (e != cudaErrorNotSupported) return e;   // strides a tensor map cannot hold: the other kernel
  }
  return a.kv.dtype == PCT_BF16 ? launch_attn_mma(p, P.bm, P.grid, s) : run_simt_r(p, P, s);
}

}  // namespace pct
