// How tree attention's work is cut up, shared by its kernels.
//
// An item is (request b, kv head h, row tile mt): up to bm rows (node, query
// head of the group) against klen = ctx_len + (last node of the tile + 1)
// tokens, in ceil(klen / BK) key tiles. Items and tiles have costs in units; the
// units of all items in order are divided evenly over the grid, so lengths from
// one token to the longest balance without the host knowing them: a block's share
// may begin and end inside items (a tile goes where its first unit is). An item inside one share is written out directly; the
// pieces of a split item go to the workspace as (unnormalised fp32 sums, row
// maximum, row sum), at most two a block (slot 0: the share's first item, slot
// 1: its last), and the join kernel adds them up in unit order, so results do
// not depend on timing.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace pct {

struct AttnParams {
  int batch, n, hq, hkv, g, d, page_size, n_pages, max_pages, words;
  float scale_log2;             // scale * log2 e
  long long qs_b, qs_n, qs_h, ks_page, ks_slot, ks_head;
  const void *q, *k, *v;
  const int32_t* table;
  const int64_t* ctx_len;
  const int32_t* count;
  const uint32_t* mask;
  void* out;
  float* lse;
  int32_t* status;
  float* po;                    // [grid][2][bm][d] pieces' sums
  float2* pml;                  // [grid][2][bm] pieces' (maximum in log2 units, sum)
  int32_t* fail;                // [grid] FAIL_* bits of each block
  int bm;                       // rows of an item
  int half;                     // units: `few` a tile of an item with at most this many
  int few, many, per_item;      // rows, `many` of one with more, `per_item` an item
  uint32_t pg_mul, pg_shift;    // t / page_size = (umulhi(t, mul) + t) >> shift
  int4* meta;                   // [grid] split item begun by the block: b (-1 none),
                                // h | rows << 10, mt, slot | last block << 1
};

namespace {

constexpr float kLn2 = 0.6931471805599453f;

struct Req {
  long long ctx;
  int n, st;                    // n = 0 when st != 0
};
__device__ __forceinline__ Req attn_req(const AttnParams& p, int b) {
  Req r;
  r.ctx = p.ctx_len[b];
  r.n = p.count ? p.count[b] : p.n;
  r.st = 0;
  if (r.n < 0 || r.n > p.n) r.st |= PCT_DEV_BAD_COUNT;
  if (r.ctx < 0 || (r.st == 0 && r.ctx > (long long)p.max_pages * p.page_size - r.n))
    r.st |= PCT_DEV_BAD_LENGTH;
  if (r.st) { r.n = 0; r.ctx = 0; }
  return r;
}

// t / page_size for 0 <= t < 2^31 without a division (round-up reciprocal of 32
// + shift bits, Granlund and Montgomery 1994)
__device__ __forceinline__ uint32_t page_of(const AttnParams& p, uint32_t t) {
  return (__umulhi(t, p.pg_mul) + t) >> p.pg_shift;
}

// Which of the 32 tokens at node offsets j .. j + 31 (negative: context) row
// `node` sees; `words` is its mask row or null for a causal chain.
__device__ __forceinline__ uint32_t seen32(const AttnParams& p, const uint32_t* words, int node,
                                           int j) {
  const int live = node - j + 1;
  if (live <= 0) return 0u;
  uint32_t bits = 0xffffffffu;
  if (words && j > -32) {
    const int w = j >> 5, sh = j & 31;
    const uint32_t lo = w < 0 ? 0xffffffffu : w < p.words ? __ldg(words + w) : 0u;
    const uint32_t hi = w + 1 < p.words ? __ldg(words + w + 1) : 0u;
    bits = __funnelshift_r(lo, hi, sh);
  }
  return live < 32 ? bits & ((1u << live) - 1u) : bits;
}

template <int BK>
struct Sched {
  // tokens that the rows of tile mt see at most
  static __device__ __forceinline__ int klen(const AttnParams& p, const Req& r, int mt) {
    const int last = min(r.n, ((mt + 1) * p.bm - 1) / p.g + 1);
    return (int)r.ctx + last;
  }
  static __device__ __forceinline__ int row_tiles(const AttnParams& p, const Req& r) {
    return (r.n * p.g + p.bm - 1) / p.bm;
  }
  static __device__ long long head_units(const AttnParams& p, const Req& r) {
    const int nm = row_tiles(p, r);
    long long s = 0;
    for (int mt = 0; mt < nm; ++mt) s += item_units(p, r, mt);
    return s;
  }
  static __device__ __forceinline__ int tiles(const AttnParams& p, const Req& r, int mt) {
    return (klen(p, r, mt) + BK - 1) / BK;
  }
  static __device__ __forceinline__ int weight(const AttnParams& p, const Req& r, int mt) {
    return min(p.bm, r.n * p.g - mt * p.bm) > p.half ? p.many : p.few;
  }
  static __device__ __forceinline__ int item_units(const AttnParams& p, const Req& r, int mt) {
    return tiles(p, r, mt) * weight(p, r, mt) + p.per_item;
  }
};

// A block's place in the schedule: its units, and the item of the first one.
struct Share {
  long long u0, u1;
  long long total, per, extra;  // per (+ 1 for the first `extra` blocks) units a block
  int b, h, mt, off;            // off: units of the item before u0
};
__device__ __forceinline__ int block_of(const Share& s, long long u) {
  const long long cut = s.extra * (s.per + 1);
  return (int)(u < cut ? u / (s.per + 1) : s.extra + (u - cut) / s.per);
}

// The walk over a share's items. All threads of a role take the same steps.
template <int BK>
struct Walk {
  typedef Sched<BK> S;
  long long u;
  int b, h, mt, off;
  Req r;
  bool fresh;
  // of the item in hand: its key tiles t0 .. t1 - 1 of nt here, rows, tokens; whether
  // that is all of it; the piece's slot where not; the join's note where it begins here
  int t0, t1, nt, rows, klen, pslot;
  bool whole;
  __device__ __forceinline__ void begin(const Share& s) {
    u = s.u0; b = s.b; h = s.h; mt = s.mt; off = s.off; fresh = true;
  }
  __device__ __forceinline__ bool next(const AttnParams& p, const Share& s, int4* begun) {
    while (u < s.u1) {
      if (fresh) r = attn_req(p, b);
      fresh = false;
      if (mt >= S::row_tiles(p, r)) { mt = 0; ++h; }
      while (h >= p.hkv || r.n == 0) { ++b; h = 0; mt = 0; r = attn_req(p, b); }
      klen = S::klen(p, r, mt);
      nt = (klen + BK - 1) / BK;
      const int w = S::weight(p, r, mt);
      // the item's own units come first, then its tiles'
      const int c = p.per_item, e = (int)min((long long)nt * w + c, off + (s.u1 - u));
      t0 = (max(off - c, 0) + w - 1) / w;
      t1 = (max(e - c, 0) + w - 1) / w;
      rows = min(p.bm, r.n * p.g - mt * p.bm);
      whole = t0 == 0 && t1 == nt;
      pslot = u == s.u0 ? 0 : 1;
      if (t0 == 0 && t1 > 0 && t1 < nt)
        *begun = make_int4(b, h | rows << 10, mt,
                           pslot | block_of(s, u - off + c + (long long)(nt - 1) * w) << 1);
      u += e - off;
      off = 0;
      ++mt;                      // (b, h, mt - 1) is the item in hand
      if (t0 < t1) return true;
    }
    return false;
  }
};

// Fills *out (shared memory); all NT threads call it.
template <int BK, int NT>
__device__ void sched_begin(const AttnParams& p, Share* out, long long* sums) {
  typedef Sched<BK> S;
  const int tid = threadIdx.x;
  const int seg = (p.batch + NT - 1) / NT;
  const int b0 = tid * seg, b1 = min(p.batch, b0 + seg);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Req r = attn_req(p, b);
    mine += S::head_units(p, r) * p.hkv;
  }
  const int lane = tid & 31, w = tid >> 5;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sums[w] = inc;
  __syncthreads();
  long long base = 0, total = 0;
#pragma unroll
  for (int k = 0; k < NT / 32; ++k) {
    if (k < w) base += sums[k];
    total += sums[k];
  }
  const long long ex = base + inc - mine;
  long long blocks = total / max(p.few, p.many);   // a whole tile at least in every part of an item
  if (blocks > gridDim.x) blocks = gridDim.x;
  if (blocks < 1) blocks = 1;
  const long long per = total / blocks, extra = total - per * blocks;
  const long long c = blockIdx.x;
  const long long u0 = c < blocks ? c * per + (c < extra ? c : extra) : total;
  const long long u1 = c < blocks ? u0 + per + (c < extra ? 1 : 0) : total;
  if (tid == 0) {
    out->u0 = u0; out->u1 = u1; out->total = total; out->per = per; out->extra = extra;
    out->b = -1; out->h = out->mt = out->off = 0;
  }
  __syncthreads();
  if (u0 < u1 && u0 >= ex && u0 < ex + mine) {
    long long at = ex;
    for (int b = b0; b < b1; ++b) {
      const Req r = attn_req(p, b);
      const long long hu = S::head_units(p, r), all = hu * p.hkv;
      if (u0 < at + all) {
        long long rest = u0 - at;
        const int h = (int)(rest / hu);
        rest -= h * hu;
        int mt = 0;
        for (;; ++mt) {
          const int t = S::item_units(p, r, mt);
          if (rest < t) break;
          rest -= t;
        }
        out->b = b; out->h = h; out->mt = mt; out->off = (int)rest;
        break;
      }
      at += all;
    }
  }
  __syncthreads();
}

// Rows at or past count (and all rows of a refused request) to 0 and -inf. Requests
// are spread over the grid, several blocks a request where there are more blocks.
template <typename T>
__device__ void attn_zero(const AttnParams& p, int tid, int threads) {
  const int parts = max(1, (int)gridDim.x / p.batch);
  for (int task = blockIdx.x; task < p.batch * parts; task += gridDim.x) {
    const int b = task % p.batch, part = task / p.batch;
    const Req r = attn_req(p, b);
    const long long r0 = ((long long)b * p.n + r.n) * p.hq, r1 = ((long long)b * p.n + p.n) * p.hq;
    const int vec = p.d * (int)sizeof(T) / 16;
    uint4* o = static_cast<uint4*>(p.out);
    for (long long i = r0 * vec + part * threads + tid; i < r1 * vec; i += (long long)parts * threads)
      o[i] = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (long long i = r0 + part * threads + tid; i < r1; i += (long long)parts * threads)
        p.lse[i] = neg_inf();
  }
}

// A block's report in p.fail.
constexpr int FAIL_TIMEOUT = 1, FAIL_PAGE = 2;

// Status words, by the join: block tables are looked over again only if some block
// met a bad page. All threads of the blocks with blockIdx.y == 0 call it.
__device__ __forceinline__ void attn_status(const AttnParams& p) {
  int any = 0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += blockDim.x) any |= p.fail[i];
  const int late = __syncthreads_or(any & FAIL_TIMEOUT), page = __syncthreads_or(any & FAIL_PAGE);
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    const Req r = attn_req(p, b);
    int bad = 0;
    if (page && r.n > 0) {
      const int32_t* row = p.table + (long long)b * p.max_pages;
      const int e = (int)((r.ctx + r.n - 1) / p.page_size);
      for (int k = threadIdx.x; k <= e; k += blockDim.x) bad |= row[k] < 0 || row[k] >= p.n_pages;
    }
    if (page) bad = __syncthreads_or(bad);
    if (threadIdx.x == 0)
      p.status[b] = r.st | (bad ? PCT_DEV_BAD_PAGE : 0) | (late ? PCT_DEV_TIMEOUT : 0);
  }
}

// 1 / sum and the log-sum-exp of a row (maximum in log2 units): 0 and -inf for a
// row that sees nothing, NaN where a score was
__device__ __forceinline__ float inverse(float l) {
  return l > 0.f ? 1.f / l : (l == l ? 0.f : l);
}
__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.f ? (m + __log2f(l)) * kLn2 : (l == l ? neg_inf() : l);
}

__device__ __forceinline__ void store_out(float* p, float4 v) {
  *reinterpret_cast<float4*>(p) = v;
}
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 w;
  w.x = *reinterpret_cast<uint32_t*>(&a);
  w.y = *reinterpret_cast<uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = w;
}

// A row's pieces, in unit order, with the running maximum. JOIN_AHEAD pieces' maxima,
// sums and values are asked for together (unconditionally: past the last piece the
// last one again, without weight), so the join waits for memory a few times and not
// twice a piece.
constexpr int JOIN_AHEAD = 8;
struct JoinState {
  float m, l;
  __device__ __forceinline__ void begin() { m = neg_inf(); l = 0.f; }
  // the factors of the sums so far and of the new piece
  __device__ __forceinline__ float2 add(float2 a) {
    const float mn = fmaxf(m, a.x), ref = mn == neg_inf() ? 0.f : mn;
    const float2 f = make_float2(ex2(m - ref), ex2(a.x - ref));
    l = l * f.x + a.y * f.y;
    m = mn;
    return f;
  }
};
__device__ __forceinline__ void join_add(float4& acc, float4 x, float2 f) {
  acc.x = fmaf(x.x, f.y, acc.x * f.x);
  acc.y = fmaf(x.y, f.y, acc.y * f.x);
  acc.z = fmaf(x.z, f.y, acc.z * f.x);
  acc.w = fmaf(x.w, f.y, acc.w * f.x);
}

// Joins the pieces of the split item that block blockIdx.x of the attention
// kernel began: one warp a row, its lanes over head_dim.
template <typename T, int BM, bool WIDE>   // WIDE: head_dim above 128
__global__ void __launch_bounds__(128) attn_join_kernel(AttnParams p) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x;
  const int4 m = p.meta[c];
  if (blockIdx.y == 0) attn_status(p);
  if (m.x < 0) return;
  const int b = m.x, h = m.y & 1023, rows = m.y >> 10, mt = m.z, slot = m.w & 1, last = m.w >> 1;
  const int lane = threadIdx.x & 31;
  const int d0 = lane * 4 < p.d ? lane * 4 : 0, d1 = lane * 4 + 128 < p.d ? lane * 4 + 128 : 0;
  for (int i = blockIdx.y * 4 + (threadIdx.x >> 5); i < rows; i += gridDim.y * 4) {
    JoinState st;
    st.begin();
    float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int k0 = c; k0 <= last; k0 += JOIN_AHEAD) {
      float2 a[JOIN_AHEAD];
      float4 x[JOIN_AHEAD], y[JOIN_AHEAD];
#pragma unroll
      for (int j = 0; j < JOIN_AHEAD; ++j) {
        const int k = min(k0 + j, last);
        const long long at = ((long long)k * 2 + (k == c ? slot : 0)) * BM + i;
        a[j] = p.pml[at];
        x[j] = *reinterpret_cast<const float4*>(p.po + at * p.d + d0);
        if (WIDE) y[j] = *reinterpret_cast<const float4*>(p.po + at * p.d + d1);
      }
#pragma unroll
      for (int j = 0; j < JOIN_AHEAD; ++j) {
        if (k0 + j > last) break;
        const float2 f = st.add(a[j]);
        join_add(acc[0], x[j], f);
        if (WIDE) join_add(acc[1], y[j], f);
      }
    }
    const int row = mt * BM + i, node = row / p.g, qh = h * p.g + row % p.g;
    const long long o = ((long long)b * p.n + node) * p.hq + qh;
    const float inv = inverse(st.l);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int d = j * 128 + lane * 4;
      if (d < p.d)
        store_out(static_cast<T*>(p.out) + o * p.d + d,
                  make_float4(acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv));
    }
    if (p.lse && lane == 0) p.lse[o] = lse_of(st.m == neg_inf() ? 0.f : st.m, st.l);
  }
}

}  // namespace
}  // namespace pct
