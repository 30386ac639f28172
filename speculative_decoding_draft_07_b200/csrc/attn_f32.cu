// Tree attention for fp32 caches: products on the tensor cores in three TF32 parts.
//
// Each factor x is split into hi = x rounded to TF32 (11 bits) and lo = x - hi, of
// which the product reads 11 bits, and a product is hi hi + hi lo + lo hi with fp32
// accumulation: off by at most 5 * 2^-22 of |x y|, the size of an fp32 sum's own
// rounding over twenty terms. On the FP32 pipes the same tiles took 2600 instructions a warp for 32 keys
// x 32 rows and kept shared memory 60% busy (4 requests x 32 nodes, 8 heads of 64
// over up to 1777 tokens: 40 us); this takes 28. Decode of 32 requests over up to 16384
// tokens reads 4.5 TB/s: DRAM is at 50%, tensor pipe 39%, integer pipe 30%, issue 47%, so
// nothing is full; with two warps a scheduler the chains of split and product wait for
// themselves. From some ten rows on the products bound it.
// The block is that of the bf16 kernel: four warps, WM of 16 rows each, the others
// splitting a tile's keys, each with its own running maximum, sum and accumulator;
// tiles of 64 keys (32 above head_dim 64) in a ring of asynchronous copies. Rows lie
// DP + 4 floats apart, so that the matrix loads of K (8 rows x 4 floats a matrix) and
// the scalar loads of V (two neighbouring keys x 8 columns) find no bank conflicts. The
// weights' matrix layout pairs keys 2t and 2t + 1 where the next product wants t and
// t + 4; the order of keys in a sum is free, so V is read in the weights' order.
#include <type_traits>

#include "attn_warp.cuh"

namespace pct {
namespace {

constexpr int kF32Threads = 128;

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x as hi (TF32, to nearest) + lo (the rest; the product reads its upper 19 bits). An
// infinite x gives lo = NaN, and a finite |x| from 0x7f7ff000 (3.402e38) on is rounded up
// to hi = inf, lo = -inf; both make every product NaN. The callers look for NaN and take
// such scores and sums again.
struct Part { uint32_t hi, lo; };
__device__ __forceinline__ Part split(uint32_t x) {
  Part p;
  p.hi = (x + 0x1000u) & 0xffffe000u;
  p.lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(p.hi));
  return p;
}
struct PartA {
  uint32_t hi[4], lo[4];
  __device__ __forceinline__ void set(int j, uint32_t x) {
    const Part p = split(x);
    hi[j] = p.hi; lo[j] = p.lo;
  }
};
// c += a b in three parts, the small ones (into e, which may be c) first
__device__ __forceinline__ void mma_f32(float (&c)[4], float (&e)[4], const PartA& a,
                                        const Part& b0, const Part& b1) {
  mma_tf32(e, a.lo, b0.hi, b1.hi);
  mma_tf32(e, a.hi, b0.lo, b1.lo);
  mma_tf32(c, a.hi, b0.hi, b1.hi);
}

// The product of weights a >= 0 with any values b: hi of a very large one is cut off where
// rounding would make it infinite, and an infinity is hi alone, which only a's hi meets (a's
// lo may be 0 or negative). Other values come out as by split and mma_f32, bit for bit.
struct PartB { Part p; uint32_t lo_hi; };              // lo_hi: hi as a's lo meets it
__device__ __forceinline__ PartB split_any(uint32_t x) {
  const uint32_t mag = x & 0x7fffffffu;
  PartB r;
  r.p = split(x);
  if (mag >= 0x7f7ff000u && mag <= 0x7f800000u) {
    r.p.hi = mag == 0x7f800000u ? x : x & 0xffffe000u;
    r.p.lo = mag == 0x7f800000u ? 0u
                                : __float_as_uint(__uint_as_float(x) - __uint_as_float(r.p.hi));
  }
  r.lo_hi = mag == 0x7f800000u ? 0u : r.p.hi;
  return r;
}
__device__ __forceinline__ void mma_any(float (&c)[4], const PartA& a, const PartB& b0,
                                        const PartB& b1) {
  mma_tf32(c, a.lo, b0.lo_hi, b1.lo_hi);
  mma_tf32(c, a.hi, b0.p.lo, b1.p.lo);
  mma_tf32(c, a.hi, b0.p.hi, b1.p.hi);
}

template <int DP, int WM> struct F32Shape {
  static constexpr int BK = DP == 64 ? 64 : 32;
  // two blocks an SM; a third stage where the cache's bytes bound (few rows)
  static constexpr int STAGES = DP == 256 || WM > 1 ? 2 : 3;
  static constexpr int PITCH = DP + 4;                 // floats from row to row
  static constexpr int TILE = BK * PITCH * 4;          // bytes of a K (or V) tile
  static constexpr int MINB = DP == 256 ? 1 : 2;
};

// DP: head_dim rounded up to 64, 128 or 256 (the rest is zero).
template <int DP, int WM>
__global__ void __launch_bounds__(kF32Threads, F32Shape<DP, WM>::MINB) attn_f32_kernel(AttnParams p) {
  constexpr int WK = 4 / WM, BM = 16 * WM, BK = F32Shape<DP, WM>::BK, NT = kF32Threads;
  constexpr int KW = BK / WK;                          // keys of a warp
  constexpr int CH = DP / 4;                           // 16-byte pieces a row
  constexpr int STAGES = F32Shape<DP, WM>::STAGES, TILE = F32Shape<DP, WM>::TILE;
  constexpr int RB = F32Shape<DP, WM>::PITCH * 4;          // bytes from row to row
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Share share;
  __shared__ long long sums[NT / 32];
  // per tile (ring of four): where its tokens' rows lie, -1 for none, and the keys
  // whose page is bad. Worked out a tile ahead of the copies, one thread a token, so
  // that no copy waits for the block table.
  __shared__ long long where[4][BK];
  __shared__ unsigned long long gone[4];
  __shared__ float2 ml[WK][BM];
  unsigned char* Qs = smem;                            // [BM][PITCH]
  unsigned char* ring = smem + BM * RB;                // [STAGES][K, V][BK][PITCH]
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
      const bool in = c * 4 < p.d;
      const uint32_t kd = sm_addr(ring + st * 2 * TILE), vd = kd + TILE;
#pragma unroll
      for (int i = 0; i < BK / RS; ++i) {
        const int rr = i * RS + r0;
        const uint32_t at = rr * RB + c * 16;
        const long long w = where[t & 3][rr];
        const bool on = in && w >= 0;
        const long long off = on ? w + c * 4 : 0;
        cp16(kd + at, kb + off, on ? 16 : 0);
        cp16(vd + at, vb + off, on ? 16 : 0);
      }
    };

    const int ra = wm * 16 + (lane >> 2);
    const uint32_t qa = sm_addr(Qs) + (wm * 16 + (lane & 15)) * RB + (lane >> 4) * 16;
    float acc[DP / 8][4], m[2], l[2];
    // The item's tiles; whether a sum of P V came out NaN although its row's scores did not.
    // That is an infinite or very large V: the item is gone through again with mma_any, and
    // what was not NaN stays as it was. (Two copies of the loop: a call or a branch to the
    // other products inside one made fp32 decode 40% slower; this leaves it as it was, takes
    // 0.8 of 27 us with 4 requests x 32 nodes and, at worst, 6 of 111 us at head_dim 256 with
    // 17 to 32 rows.)
    auto tiles = [&](auto again) -> bool {
      __syncthreads();                                   // the last item's buffers are free
#pragma unroll
      for (int i = 0; i < STAGES; ++i)
        if (t0 + i < t1) find_tile(t0 + i);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < BM * CH / NT; ++i) {
        const int rr = (i * NT + tid) / CH, c = tid % CH;
        const float* src = static_cast<const float*>(p.q);
        int bytes = 0;
        if (rr < rows && c * 4 < p.d) {
          const int row = row0 + rr, node = row / p.g, qh = h * p.g + (row - node * p.g);
          src += b * p.qs_b + node * p.qs_n + qh * p.qs_h + c * 4;
          bytes = 16;
        }
        cp16(sm_addr(Qs) + rr * RB + c * 16, src, bytes);
      }
#pragma unroll
      for (int i = 0; i < STAGES - 1; ++i) {
        if (t0 + i < t1) load_tile(t0 + i);
        cp_commit();
      }
      // this thread's rows and their nodes
      int node[2];
      const uint32_t* words[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rr = ra + i * 8;
        node[i] = rr < rows ? (row0 + rr) / p.g : -0x40000000;
        words[i] = p.mask && rr < rows ? p.mask + ((long long)b * p.n + node[i]) * p.words : nullptr;
      }
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
        const int st = (t - t0) % STAGES;
        const uint32_t kd = sm_addr(ring + st * 2 * TILE);
        const uint32_t* Vs = reinterpret_cast<const uint32_t*>(ring + (st * 2 + 1) * TILE);
        // few keys a warp: more accumulators, so that products do not wait for each other
        constexpr int E = KW <= 16 ? 2 : 1;
        float s[KW / 8][4], s2[KW / 8][4], e[KW / 8][E][4];
#pragma unroll
        for (int i = 0; i < KW / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j] = e[i][0][j] = e[i][E - 1][j] = 0.f;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {              // 16 columns: two steps of 8
          PartA a[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t x[4];
            ldsm4(qa + (2 * k + q) * 32, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) a[q].set(j, x[j]);
          }
#pragma unroll
          for (int i = 0; i < KW / 8; ++i) {
            uint32_t x[4];                               // columns 0-3, 4-7, 8-11, 12-15 of 8 keys
            ldsm4(kd + (wk * KW + i * 8 + (lane & 7)) * RB + k * 64 + (lane >> 3) * 16, x);
            mma_f32(s[i], e[i][0], a[0], split(x[0]), split(x[1]));
            mma_f32(s2[i], e[i][E - 1], a[1], split(x[2]), split(x[3]));
          }
        }
#pragma unroll
        for (int i = 0; i < KW / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = (s[i][j] + s2[i][j]) + (E == 2 ? e[i][0][j] + e[i][E - 1][j] : e[i][0][j]);
        // An infinite or very large key (or query) makes NaN of the parts where the score need
        // not be: scores that are NaN are taken again as plain sums, and only those, so that a
        // key changes no row that does not see it. (Rare.)
        bool bad = false;
#pragma unroll
        for (int i = 0; i < KW / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) bad |= !(s[i][j] == s[i][j]);
        if (__any_sync(0xffffffffu, bad)) {
          const float* Kf = reinterpret_cast<const float*>(ring + st * 2 * TILE);
          const float* Qf = reinterpret_cast<const float*>(Qs);
#pragma unroll
          for (int i = 0; i < KW / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float* kr = Kf + (wk * KW + i * 8 + 2 * (lane & 3) + (j & 1)) * (RB / 4);
              const float* qr = Qf + (ra + (j >> 1) * 8) * (RB / 4);
              float x = 0.f;
              for (int d = 0; d < p.d; ++d) x = fmaf(qr[d], kr[d], x);
              s[i][j] = s[i][j] == s[i][j] ? s[i][j] : x;
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
        // A tile's sum of P V is begun afresh and added to the accumulator by an fp32 add:
        // the matrix unit cuts its sums off instead of rounding them, which over a long
        // chain of tiles would add up to one side.
        PartA a[KW / 8];                                 // keys 2t and 2t + 1 of each eight
#pragma unroll
        for (int i = 0; i < KW / 8; ++i) {
          a[i].set(0, __float_as_uint(s[i][0]));
          a[i].set(1, __float_as_uint(s[i][2]));
          a[i].set(2, __float_as_uint(s[i][1]));
          a[i].set(3, __float_as_uint(s[i][3]));
        }
        const uint32_t* vr = Vs + (wk * KW + 2 * (lane & 3)) * (RB / 4) + (lane >> 2);
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < KW / 8; ++i) {
            const uint32_t v0 = vr[i * 8 * (RB / 4) + j * 8], v1 = vr[(i * 8 + 1) * (RB / 4) + j * 8];
            if constexpr (decltype(again)::value) mma_any(c, a[i], split_any(v0), split_any(v1));
            else mma_f32(c, c, a[i], split(v0), split(v1));
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[j][q] += c[q];
        }
        if (lost) {                                      // rare: clear the mark for the stage's next tile
          __syncthreads();
          if (tid == 0) gone[t & 3] = 0;
        }
      }
      cp_wait<0>();
      bool lost_sum = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if ((lane & 3) == 0) ml[wk][ra + i * 8] = make_float2(m[i], l[i]);
        bool nan = false;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j)
          nan |= !(acc[j][2 * i] == acc[j][2 * i]) || !(acc[j][2 * i + 1] == acc[j][2 * i + 1]);
        lost_sum |= nan && l[i] == l[i];
      }
      return lost_sum;
    };
    if (__syncthreads_or(tiles(std::false_type()))) {
      tiles(std::true_type());
      __syncthreads();
    }
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
        store_out(static_cast<float*>(p.out) + o * p.d + c,
                  make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
        if (p.lse && c == 0) p.lse[o] = lse_of(ref, sum);
      } else {
        const long long at = ((long long)blockIdx.x * 2 + slot) * BM + rr;
        *reinterpret_cast<float4*>(p.po + at * p.d + c) = x;
        if (c == 0) p.pml[at] = make_float2(mx, sum);
      }
    }
  }
  attn_zero<float>(p, tid, NT);
  __syncthreads();
  if (tid == 0) {
    p.meta[blockIdx.x] = begun;
    p.fail[blockIdx.x] = lost_page;
  }
}

template <int DP, int WM>
cudaError_t run_f32(const AttnParams& p, int grid, cudaStream_t s) {
  constexpr int BM = 16 * WM;
  constexpr size_t smem = BM * F32Shape<DP, WM>::PITCH * 4 + F32Shape<DP, WM>::STAGES * 2 * F32Shape<DP, WM>::TILE;
  static_assert(4 / WM * BM * (DP + 8) * 4 <= F32Shape<DP, WM>::STAGES * 2 * F32Shape<DP, WM>::TILE,
                "the items' end reuses the ring");
  cudaError_t e = cudaFuncSetAttribute(attn_f32_kernel<DP, WM>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  {
    TraceScope t(s, "attn_f32");
    e = launch_pdl(attn_f32_kernel<DP, WM>, dim3(grid), dim3(kF32Threads), smem, s, 1, p);
  }
  if (e != cudaSuccess) return e;
  TraceScope t(s, "attn_join");
  return launch_pdl(attn_join_kernel<float, BM, DP == 256>, dim3(grid, (BM + 3) / 4), dim3(128), 0, s,
                    1, p);
}
template <int DP>
cudaError_t run_f32_m(const AttnParams& p, int wm, int grid, cudaStream_t s) {
  if (wm == 1) return run_f32<DP, 1>(p, grid, s);
  if (wm == 2) return run_f32<DP, 2>(p, grid, s);
  return run_f32<DP, 4>(p, grid, s);
}

}  // namespace

int attn_f32_blocks(int d) { return d > 128 ? 1 : 2; }

cudaError_t launch_attn_f32(const AttnParams& p, int bm, int grid, cudaStream_t s) {
  const int wm = bm / 16;
  if (p.d <= 64) return run_f32_m<64>(p, wm, grid, s);
  if (p.d <= 128) return run_f32_m<128>(p, wm, grid, s);
  return run_f32_m<256>(p, wm, grid, s);
}

}  // namespace pct
