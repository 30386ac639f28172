// Tree attention for bf16 caches and few rows, any page size (mma.sync).
//
// It takes calls of up to 32 rows (nodes x query heads of a group) a KV head, and
// larger ones whose pages (no multiple of 8 tokens), strides or scale (not positive)
// the tcgen05 kernel cannot take. With so few rows against each key the cache's bytes
// bound it and the warp-level matrix instructions keep up: 32 decode requests over up
// to 32768 tokens, 8 heads of 128, take 340-347 us on the device (6.5-6.6 TB/s; a copy, which
// also writes, reaches 6.46). A block of four
// warps is WM x WK: WM warps of 16 rows each, the others splitting the keys of a
// tile (one row group: four warps on 16 keys each). Every warp keeps its own
// running maximum, sum and 16 x head_dim accumulator in registers; they meet only
// at the end of an item. Tiles of 64 keys arrive by 16-byte asynchronous copies
// in a ring of three stages (96 KB for head_dim 128, two blocks an SM), rows in
// 16-byte pieces swizzled by row so that the matrix loads find no bank conflicts.
#include "attn_warp.cuh"

namespace pct {
namespace {

constexpr int kMmaBK = 64;
constexpr int kMmaThreads = 128;

__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}

template <int DP> struct MmaShape {
  static constexpr int STAGES = 3;
  static constexpr int TILE = kMmaBK * DP * 2;         // bytes of a K (or V) tile
  static constexpr int MINB = DP == 256 ? 1 : 2;
};

// DP: head_dim rounded up to 64, 128 or 256 (the rest is zero).
template <int DP, int WM>
__global__ void __launch_bounds__(kMmaThreads, MmaShape<DP>::MINB) attn_mma_kernel(AttnParams p) {
  constexpr int WK = 4 / WM, BM = 16 * WM, BK = kMmaBK, NT = kMmaThreads;
  constexpr int KW = BK / WK;                          // keys of a warp
  constexpr int CH = DP / 8;                           // 16-byte pieces a row
  constexpr int STAGES = MmaShape<DP>::STAGES, TILE = MmaShape<DP>::TILE;
  constexpr bool QREG = DP <= 128;                     // Q fragments stay in registers
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Share share;
  __shared__ long long sums[NT / 32];
  // per tile (ring of four): where its tokens' rows lie, -1 for none, and the keys
  // whose page is bad. Worked out a tile ahead of the copies, one thread a token, so
  // that no copy waits for the block table.
  __shared__ long long where[4][BK];
  __shared__ unsigned long long gone[4];
  __shared__ float2 ml[WK][BM];
  unsigned char* Qs = smem;                            // [BM][DP]
  unsigned char* ring = smem + BM * DP * 2;            // [STAGES][K, V][BK][DP]
  float* obuf = reinterpret_cast<float*>(ring);        // [WK][BM][DP + 8] at an item's end
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wm = warp % WM, wk = warp / WM;
  __shared__ int lost_page;
  if (tid < 4) gone[tid] = 0;
  if (tid == 0) lost_page = 0;
  pdl_wait();
  pdl_trigger();
  sched_begin<BK, NT>(p, &share, sums);
  int4 begun = make_int4(-1, 0, 0, 0);

  Walk<BK> w;
  w.begin(share);
  while (w.next(p, share, &begun)) {
    const Req r = w.r;
    const int b = w.b, h = w.h, t0 = w.t0, t1 = w.t1, klen = w.klen, rows = w.rows;
    const int row0 = (w.mt - 1) * BM;
    const int ctx = (int)r.ctx;
    const int32_t* table = p.table + (long long)b * p.max_pages;
    const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(p.k) + h * p.ks_head;
    const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(p.v) + h * p.ks_head;

    auto find_tile = [&](int t) {
      if (tid >= BK) return;
      const int tok = t * BK + tid;
      long long off = -1;
      if (tok < klen) {
        const uint32_t col = page_of(p, tok);
        const int page = __ldg(table + col);
        if (page >= 0 && page < p.n_pages)
          off = page * p.ks_page + (tok - (int)col * p.page_size) * p.ks_slot;
        else {
          atomicOr(&gone[t & 3], 1ull << tid);
          lost_page = FAIL_PAGE;
        }
      }
      where[t & 3][tid] = off;
    };
    auto load_tile = [&](int t) {
      const int st = (t - t0) % STAGES;
      constexpr int RS = NT / CH;                      // rows a pass
      const int c = tid % CH, r0 = tid / CH;
      const bool in = c * 8 < p.d;
      const uint32_t kd = sm_addr(ring + st * 2 * TILE), vd = kd + TILE;
#pragma unroll
      for (int i = 0; i < BK / RS; ++i) {
        const int rr = i * RS + r0;
        const uint32_t at = rr * (DP * 2) + ((c ^ (rr & 7)) << 4);
        const long long w = where[t & 3][rr];
        const bool on = in && w >= 0;
        const long long off = on ? w + c * 8 : 0;
        cp16(kd + at, kb + off, on ? 16 : 0);
        cp16(vd + at, vb + off, on ? 16 : 0);
      }
    };

    __syncthreads();                                   // the last item's buffers are free
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
      if (t0 + i < t1) find_tile(t0 + i);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < BM * CH / NT; ++i) {
      const int rr = (i * NT + tid) / CH, c = tid % CH;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q);
      int bytes = 0;
      if (rr < rows && c * 8 < p.d) {
        const int row = row0 + rr, node = row / p.g, qh = h * p.g + (row - node * p.g);
        src += b * p.qs_b + node * p.qs_n + qh * p.qs_h + c * 8;
        bytes = 16;
      }
      cp16(sm_addr(Qs) + rr * (DP * 2) + ((c ^ (rr & 7)) << 4), src, bytes);
    }
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      if (t0 + i < t1) load_tile(t0 + i);
      cp_commit();
    }
    // this thread's rows and their nodes
    const int ra = wm * 16 + (lane >> 2);
    int node[2];
    const uint32_t* words[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = ra + i * 8;
      node[i] = rr < rows ? (row0 + rr) / p.g : -0x40000000;
      words[i] = p.mask && rr < rows ? p.mask + ((long long)b * p.n + node[i]) * p.words : nullptr;
    }
    const uint32_t qa = sm_addr(Qs) + (wm * 16 + (lane & 15)) * (DP * 2);
    uint32_t qf[QREG ? DP / 16 : 1][4];
    float acc[DP / 8][4], m[2], l[2];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    m[0] = m[1] = neg_inf();
    l[0] = l[1] = 0.f;

    for (int t = t0; t < t1; ++t) {
      cp_wait<STAGES - 2>();
      __syncthreads();
      if (t + STAGES - 1 < t1) load_tile(t + STAGES - 1);
      cp_commit();
      if (t + STAGES < t1) find_tile(t + STAGES);
      if (QREG && t == t0) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) ldsm4(qa + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4), qf[QREG ? k : 0]);
      }
      const int st = (t - t0) % STAGES;
      const uint32_t kd = sm_addr(ring + st * 2 * TILE), vd = kd + TILE;
      float s[KW / 8][4];
#pragma unroll
      for (int i = 0; i < KW / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
        uint32_t a[4];
        if (QREG) {
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j] = qf[QREG ? k : 0][j];
        } else {
          ldsm4(qa + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4), a);
        }
#pragma unroll
        for (int i = 0; i < KW / 16; ++i) {
          uint32_t x[4];
          const int key = wk * KW + i * 16 + (lane & 7) + ((lane >> 4) << 3);
          ldsm4(kd + key * (DP * 2) + (((2 * k + ((lane >> 3) & 1)) ^ (lane & 7)) << 4), x);
          mma_bf16(s[2 * i], a, x[0], x[1]);
          mma_bf16(s[2 * i + 1], a, x[2], x[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < KW / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] *= p.scale_log2;
      const int key0 = t * BK + wk * KW;               // the warp's first token
      const unsigned long long lost = gone[t & 3];
      if (key0 + KW > ctx || lost) {                   // nodes, the end, or a bad page
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int w = 0; w < (KW + 31) / 32; ++w) {
            uint32_t bits = seen32(p, words[i], node[i], key0 + w * 32 - ctx);
            bits &= ~(uint32_t)(lost >> (wk * KW + w * 32));
#pragma unroll
            for (int j = 0; j < 4 && w * 4 + j < KW / 8; ++j) {
              const uint32_t two = bits >> (j * 8 + 2 * (lane & 3));
              if (!(two & 1u)) s[w * 4 + j][2 * i] = neg_inf();
              if (!(two & 2u)) s[w * 4 + j][2 * i + 1] = neg_inf();
            }
          }
        }
      }
      float mn[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = s[0][2 * i];
#pragma unroll
        for (int j = 0; j < KW / 8; ++j) x = fmaxf(x, fmaxf(s[j][2 * i], s[j][2 * i + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        mn[i] = fmaxf(m[i], x);
      }
      if (__any_sync(0xffffffffu, mn[0] != m[0] || mn[1] != m[1])) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = mn[i] == neg_inf() ? 1.f : ex2(m[i] - mn[i]);
          l[i] *= f;
          m[i] = mn[i];
#pragma unroll
          for (int j = 0; j < DP / 8; ++j) {
            acc[j][2 * i] *= f;
            acc[j][2 * i + 1] *= f;
          }
        }
      }
      const float ref[2] = {m[0] == neg_inf() ? 0.f : m[0], m[1] == neg_inf() ? 0.f : m[1]};
#pragma unroll
      for (int j = 0; j < KW / 8; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s[j][2 * i] = ex2(s[j][2 * i] - ref[i]);
          s[j][2 * i + 1] = ex2(s[j][2 * i + 1] - ref[i]);
          l[i] += s[j][2 * i] + s[j][2 * i + 1];
        }
      // the weights enter the second product as bf16 (off by at most 2^-8 each, the
      // matrix instruction's operand type); their sum above is that of the fp32 values
#pragma unroll
      for (int i = 0; i < KW / 16; ++i) {
        const uint32_t a[4] = {pack_bf16(s[2 * i][0], s[2 * i][1]), pack_bf16(s[2 * i][2], s[2 * i][3]),
                               pack_bf16(s[2 * i + 1][0], s[2 * i + 1][1]),
                               pack_bf16(s[2 * i + 1][2], s[2 * i + 1][3])};
        const int key = wk * KW + i * 16 + (lane & 15);
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) {
          uint32_t x[4];
          ldsm4t(vd + key * (DP * 2) + (((2 * j + (lane >> 4)) ^ (lane & 7)) << 4), x);
          mma_bf16(acc[2 * j], a, x[0], x[1]);
          mma_bf16(acc[2 * j + 1], a, x[2], x[3]);
        }
      }
      if (lost) {                                      // rare: clear the mark for the stage's next tile
        __syncthreads();
        if (tid == 0) gone[t & 3] = 0;
      }
    }
    cp_wait<0>();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if ((lane & 3) == 0) ml[wk][ra + i * 8] = make_float2(m[i], l[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = neg_inf();
#pragma unroll
      for (int k = 0; k < WK; ++k) mx = fmaxf(mx, ml[k][ra + i * 8].x);
      const float f = mx == neg_inf() ? 0.f : ex2(m[i] - mx);
      float* o = obuf + (wk * BM + ra + i * 8) * (DP + 8) + 2 * (lane & 3);
#pragma unroll
      for (int j = 0; j < DP / 8; ++j)
        *reinterpret_cast<float2*>(o + j * 8) = make_float2(acc[j][2 * i] * f, acc[j][2 * i + 1] * f);
    }
    __syncthreads();
    const bool whole = w.whole;
    const int slot = w.pslot;
    const int v4 = p.d / 4;
    for (int i = tid; i < rows * v4; i += NT) {
      const int rr = i / v4, c = (i - rr * v4) * 4;
      float mx = neg_inf(), sum = 0.f;
#pragma unroll
      for (int k = 0; k < WK; ++k) mx = fmaxf(mx, ml[k][rr].x);
      const float ref = mx == neg_inf() ? 0.f : mx;
#pragma unroll
      for (int k = 0; k < WK; ++k) sum += ml[k][rr].y * ex2(ml[k][rr].x - ref);
      float4 x = *reinterpret_cast<const float4*>(obuf + rr * (DP + 8) + c);
#pragma unroll
      for (int k = 1; k < WK; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(obuf + (k * BM + rr) * (DP + 8) + c);
        x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
      }
      if (whole) {
        const int row = row0 + rr, nd = row / p.g, qh = h * p.g + (row - nd * p.g);
        const long long o = ((long long)b * p.n + nd) * p.hq + qh;
        const float inv = inverse(sum);
        store_out(static_cast<__nv_bfloat16*>(p.out) + o * p.d + c,
                  make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
        if (p.lse && c == 0) p.lse[o] = lse_of(ref, sum);
      } else {
        const long long at = ((long long)blockIdx.x * 2 + slot) * BM + rr;
        *reinterpret_cast<float4*>(p.po + at * p.d + c) = x;
        if (c == 0) p.pml[at] = make_float2(mx, sum);
      }
    }
  }
  attn_zero<__nv_bfloat16>(p, tid, NT);
  __syncthreads();
  if (tid == 0) {
    p.meta[blockIdx.x] = begun;
    p.fail[blockIdx.x] = lost_page;
  }
}

template <int DP, int WM>
cudaError_t run_mma(const AttnParams& p, int grid, cudaStream_t s) {
  constexpr int BM = 16 * WM;
  constexpr size_t smem = BM * DP * 2 + MmaShape<DP>::STAGES * 2 * MmaShape<DP>::TILE;
  static_assert(4 / WM * BM * (DP + 8) * 4 <= MmaShape<DP>::STAGES * 2 * MmaShape<DP>::TILE,
                "the items' end reuses the ring");
  cudaError_t e = cudaFuncSetAttribute(attn_mma_kernel<DP, WM>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  {
    TraceScope t(s, "attn_mma");
    e = launch_pdl(attn_mma_kernel<DP, WM>, dim3(grid), dim3(kMmaThreads), smem, s, 1, p);
  }
  if (e != cudaSuccess) return e;
  TraceScope t(s, "attn_join");
  return launch_pdl(attn_join_kernel<__nv_bfloat16, BM, DP == 256>, dim3(grid, (BM + 3) / 4), dim3(128), 0, s,
                    1, p);
}
template <int DP>
cudaError_t run_mma_m(const AttnParams& p, int wm, int grid, cudaStream_t s) {
  if (wm == 1) return run_mma<DP, 1>(p, grid, s);
  if (wm == 2) return run_mma<DP, 2>(p, grid, s);
  return run_mma<DP, 4>(p, grid, s);
}

}  // namespace

int attn_mma_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
int attn_mma_blocks(int d) { return d > 128 ? 1 : 2; }

cudaError_t launch_attn_mma(const AttnParams& p, int bm, int grid, cudaStream_t s) {
  const int wm = bm / 16;
  if (p.d <= 64) return run_mma_m<64>(p, wm, grid, s);
  if (p.d <= 128) return run_mma_m<128>(p, wm, grid, s);
  return run_mma_m<256>(p, wm, grid, s);
}

}  // namespace pct
