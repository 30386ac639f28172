// Tree attention for bf16 caches and many rows on the tcgen05 tensor cores.
//
// Above 64 rows (nodes x query heads of a group) the two products outweigh the
// cache's bytes. One block an SM works on an item of up to 256 rows against key
// tiles of 128 tokens as two streams of 128 rows (one thread a row):
//   * warp 0: TMA producer. K and V tiles alternate through a ring of 128-byte
//     swizzled slots, each page of a tile its own box (a lane a page);
//   * warp 1, one thread: issues S_s = Q_s K^T (shared x shared) and
//     O_s += P_s V (P_s from tensor memory) of whichever stream is ready, so one
//     stream's products run under the other's softmax;
//   * warps 2-5 and 6-9: the softmax of stream 0 and 1. A thread reads its row of
//     128 scores from tensor memory, keeps the running maximum and sum, and writes
//     the weights back as bf16 over the scores.
// With more than 128 rows in an item the streams are its two row tiles and share
// every K and V tile; with fewer they take alternate key tiles of the same rows
// and are added up at the item's end (both accumulators sit in the same tensor
// memory lanes). Tensor memory: S_0, S_1 (128 columns each; P_s in the first 64
// of S_s), O_0, O_1. The accumulator is rescaled only when a row's maximum grows by
// more than 2^8 over the reference in use, which the later tiles seldom do;
// weights up to 2^8 lose nothing in fp32 sums and bf16 products.
// Every mbarrier wait is bounded; when one gives up, the roles run to the end
// without waiting, drain their copies and products, free the tensor memory, and
// the join reports PCT_DEV_TIMEOUT.
#include <cuda.h>

#include <algorithm>

#include "attn_sched.cuh"
#include "umma.cuh"

namespace pct {
namespace {

constexpr int UBM = 256;                 // rows of an item
constexpr int UBK = 128;                 // tokens of a key tile
constexpr int UTHREADS = 320;
constexpr int GONE = 4;                  // tiles whose bad-page marks are kept

template <int DP> struct UShape {
  static constexpr int HALVES = DP / 64;                   // 64-column boxes of a row
  static constexpr int QTILE = 128 * DP * 2;
  static constexpr int SLOT = UBK * DP * 2;
  static constexpr int SLOTS = 4;
  static constexpr size_t SMEM = 1024 + 2 * QTILE + SLOTS * SLOT;
};

struct UMaps {
  int rows, shift;                       // tokens of a box (a page, at most 128), its log2
  int slot_dim;                          // map axis of the token in a page: 1 or 2
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
// D += A B with A (bf16 pairs) in tensor memory
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void pair_sync() {   // both softmax groups
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

// The items of a block's share, in order. seq numbers the key tiles that the
// block loads (their ring slots follow from it).
struct Walk {
  long long u;
  int b, h, mt, t0, t1, nt, rows, klen, seq, items;
  bool split, first;
  Req r;
  __device__ void begin(const Share& s) {
    u = s.u0; b = s.b; h = s.h; mt = s.mt; t0 = s.tile; t1 = t0; nt = 0;
    seq = 0; items = 0; first = true; split = false;
    r.n = 0;
  }
  __device__ bool next(const AttnParams& p, const Share& s) {
    typedef Sched<UBM, UBK> S;
    if (!first) {
      seq += t1 - t0;
      u += t1 - t0;
      t0 = 0;
      ++mt;
      ++items;
    }
    if (u >= s.u1) return false;
    if (first) r = attn_req(p, b);
    first = false;
    if (mt >= S::row_tiles(p, r)) { mt = 0; ++h; }
    while (h >= p.hkv || r.n == 0) { ++b; h = 0; mt = 0; r = attn_req(p, b); }
    klen = S::klen(p, r, mt);
    nt = (klen + UBK - 1) / UBK;
    t1 = (int)min((long long)nt, t0 + (s.u1 - u));
    rows = min(UBM, r.n * p.g - mt * UBM);
    split = rows <= 128;
    return true;
  }
  // key tiles of stream st: first, and how many
  __device__ int start(int st) const { return split ? t0 + st : t0; }
  __device__ int step() const { return split ? 2 : 1; }
};

template <int DP>
__global__ void __launch_bounds__(UTHREADS, 1)
attn_umma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const AttnParams p, const UMaps mp) {
  typedef UShape<DP> U;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint8_t* ring = sQ + 2 * U::QTILE;
  __shared__ uint64_t full[U::SLOTS], empty[U::SLOTS], qready[2], sfull[2], pready[2], pvdone[2],
      drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ uint4 gone[GONE];
  __shared__ float2 ml[2][128];
  __shared__ Share share;
  __shared__ long long sums[UTHREADS / 32];
  volatile int* abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* err = p.fail + blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < U::SLOTS; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 2); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qready[i], 128);
      mbar_init(&sfull[i], 1);
      mbar_init(&pready[i], 128);
      mbar_init(&pvdone[i], 1);
    }
    mbar_init(&drain, 1);
    abort_word = 0;
    *err = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_slot)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  sched_begin<UBM, UBK, UTHREADS>(p, 1, &share, sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t tS = tmem, tO = tmem + 256;
  int4 begun = make_int4(-1, 0, 0, 0);

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    Walk w;
    w.begin(share);
    bool ok = true;
    uint32_t armed = 0, armed_par = 0;
    const int boxes = UBK >> mp.shift;              // boxes of a tile
    while (ok && w.next(p, share)) {
      const int32_t* table = p.table + (long long)w.b * p.max_pages;
      for (int t = w.t0; t < w.t1 && ok; ++t) {
        const int seq = w.seq + t - w.t0;
        const int tok = t * UBK + (lane << mp.shift);
        int page = -1, place = 0;
        const bool live = lane < boxes && tok < w.klen;
        if (live) {
          const uint32_t col = page_of(p, tok);
          page = __ldg(table + col);
          place = tok - (int)col * p.page_size;
          if (page >= p.n_pages) page = -1;
        }
        const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
        const uint32_t lost = __ballot_sync(0xffffffffu, live && page < 0);
        if (lane == 0) {
          uint32_t g[4] = {0, 0, 0, 0};
          for (int i = 0; lost >> i; ++i)
            if ((lost >> i) & 1)
              for (int k = i << mp.shift; k < (i + 1) << mp.shift; ++k) g[k >> 5] |= 1u << (k & 31);
          gone[seq % GONE] = make_uint4(g[0], g[1], g[2], g[3]);
        }
        const uint32_t bytes = (uint32_t)__popc(have) * mp.rows * 128u * U::HALVES;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int pos = seq * 2 + kv, slot = pos % U::SLOTS;
          const uint32_t par = (uint32_t)(pos / U::SLOTS) & 1u;
          const bool got = wait_bar(&empty[slot], par ^ 1u, abort_flag, err);
          if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
          if (lane == 0) mbar_expect_tx(&full[slot], bytes);
          __syncwarp();
          if (page >= 0) {
            const uint32_t dst = smem_u32(ring + slot * U::SLOT) + (uint32_t)(lane << mp.shift) * 128u;
            const int y = mp.slot_dim == 1 ? place : w.h, z = mp.slot_dim == 1 ? w.h : place;
#pragma unroll
            for (int hf = 0; hf < U::HALVES; ++hf)
              tma_load_4d(dst + hf * (UBK * 128), kv ? &tmV : &tmK, hf * 64, y, z, page, &full[slot]);
          }
          armed |= 1u << slot;
          armed_par = (armed_par & ~(1u << slot)) | (par << slot);
        }
      }
    }
    // every copy has landed before the block may exit
#pragma unroll
    for (int i = 0; i < U::SLOTS; ++i)
      if (armed & (1u << i)) drain_wait(&full[i], (armed_par >> i) & 1u);
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- products ----------------
      constexpr uint32_t BASE = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 4) << 24);
      constexpr uint32_t ID_QK = BASE | ((uint32_t)(UBK >> 3) << 17);
      constexpr uint32_t ID_PV = BASE | (1u << 16) | ((uint32_t)(DP >> 3) << 17);
      const uint64_t q_desc = make_desc(smem_u32(sQ), 16, 1024);
      const uint64_t k_desc = make_desc(smem_u32(ring), 16, 1024);
      const uint64_t v_desc = make_desc(smem_u32(ring), UBK * 128, 1024);
      Walk w[2];
      int t[2], qk[2] = {0, 0}, pv[2] = {0, 0};     // tile in hand; products issued
      bool live[2], turn[2] = {false, false};       // turn: S is out, P V is next
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        w[s].begin(share);
        do {
          live[s] = w[s].next(p, share);
          t[s] = live[s] ? w[s].start(s) : 0;
        } while (live[s] && t[s] >= w[s].t1);
      }
      long long t0 = clock64();
      uint32_t spins = 0;
      while (live[0] || live[1]) {
        bool moved = false;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!live[s]) continue;
          const int pos = (w[s].seq + t[s] - w[s].t0) * 2;
          if (!turn[s]) {
            const int slot = pos % U::SLOTS;
            if (!mbar_test(&full[slot], (uint32_t)(pos / U::SLOTS) & 1u)) continue;
            if (qk[s] > 0 && !mbar_test(&pvdone[s], (uint32_t)(pv[s] - 1) & 1u)) continue;
            if (!mbar_test(&qready[s], (uint32_t)w[s].items & 1u)) continue;
            tc_fence_after();
            const uint64_t qd = q_desc + (uint64_t)((s * U::QTILE) >> 4);
            const uint64_t kd = k_desc + (uint64_t)((slot * U::SLOT) >> 4);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
              const uint64_t off = (uint64_t)(((k >> 2) * (UBK * 128) + (k & 3) * 32) >> 4);
              umma_f16(tS + s * 128, qd + off, kd + off, ID_QK, k > 0);
            }
            umma_commit(&sfull[s]);
            umma_commit(&empty[slot]);
            if (w[s].split) umma_commit(&empty[slot]);
            ++qk[s];
            turn[s] = true;
          } else {
            const int slot = (pos + 1) % U::SLOTS;
            if (!mbar_test(&pready[s], (uint32_t)pv[s] & 1u)) continue;
            if (!mbar_test(&full[slot], (uint32_t)((pos + 1) / U::SLOTS) & 1u)) continue;
            tc_fence_after();
            const uint64_t vd = v_desc + (uint64_t)((slot * U::SLOT) >> 4);
            const uint32_t more = t[s] != w[s].start(s);
#pragma unroll
            for (int k = 0; k < UBK / 16; ++k)
              umma_ts(tO + s * DP, tS + s * 128 + k * 8, vd + (uint64_t)((k * 2048) >> 4), ID_PV,
                      more | (k > 0));
            umma_commit(&pvdone[s]);
            umma_commit(&empty[slot]);
            if (w[s].split) umma_commit(&empty[slot]);
            ++pv[s];
            turn[s] = false;
            t[s] += w[s].step();
            while (live[s] && t[s] >= w[s].t1) {
              live[s] = w[s].next(p, share);
              t[s] = live[s] ? w[s].start(s) : 0;
            }
          }
          moved = true;
        }
        if (moved) {
          spins = 0;
        } else if ((++spins & 255u) == 0u) {
          if (spins == 256u) t0 = clock64();
          if (*abort_flag) break;
          if (clock64() - t0 > kTimeoutCycles) {
            *abort_flag = 1;
            atomicExch(err, 1);
            break;
          }
        }
      }
      umma_commit(&drain);
      drain_wait(&drain, 0);
    }
  } else {
    // ---------------- softmax ----------------
    const int s = (warp - 2) >> 2, quad = warp & 3;
    const int tl = (warp - 2 - s * 4) * 32 + lane;       // thread of the group
    const int rr = quad * 32 + lane;                     // row of the stream = TMEM lane
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint32_t aS = tS + s * 128 + lane_base, aO = tO + s * DP + lane_base;
    const float c = p.scale_log2;
    uint8_t* myQ = sQ + s * U::QTILE;
    int done = 0;                                        // tiles of this stream so far
    auto wait = [&](uint64_t* bar, uint32_t par) {
      const bool got = wait_bar(bar, par, abort_flag, err);
      return __all_sync(0xffffffffu, got);
    };
    auto load_q = [&](const Walk& w) {
      const int base = w.mt * UBM + (w.split ? 0 : s * 128), lim = w.rows - (w.split ? 0 : s * 128);
      constexpr int CH = DP / 8;
#pragma unroll 4
      for (int i = 0; i < CH; ++i) {
        const int r0 = (i * 128 + tl) / CH, ch = tl % CH;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r0 < lim && ch * 8 < p.d) {
          const int row = base + r0, node = row / p.g, qh = w.h * p.g + (row - node * p.g);
          x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                   w.b * p.qs_b + node * p.qs_n + qh * p.qs_h +
                                                   ch * 8));
          x.x ^= p.q_sign; x.y ^= p.q_sign; x.z ^= p.q_sign; x.w ^= p.q_sign;
        }
        *reinterpret_cast<uint4*>(myQ + (ch >> 3) * (128 * 128) + r0 * 128 +
                                  (((ch & 7) ^ (r0 & 7)) << 4)) = x;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&qready[s]);
    };

    Walk w, nx;
    nx.begin(share);
    bool more = nx.next(p, share);
    if (more) load_q(nx);
    while (more) {
      w = nx;
      const int base = w.mt * UBM + (w.split ? 0 : s * 128), lim = w.rows - (w.split ? 0 : s * 128);
      const int row = base + rr;
      const bool valid = rr < lim;
      const int node = valid ? row / p.g : -0x40000000;
      const uint32_t* words =
          p.mask && valid ? p.mask + ((long long)w.b * p.n + node) * p.words : nullptr;
      const int ctx = (int)w.r.ctx;
      float m = neg_inf(), l = 0.f;
      bool any = false;
      for (int t = w.start(s); t < w.t1; t += w.step()) {
        const int seq = w.seq + t - w.t0, k0 = t * UBK;
        (void)wait(&sfull[s], (uint32_t)done & 1u);
        tc_fence_after();
        uint32_t x[128];
        tmem_issue(aS, *reinterpret_cast<uint32_t(*)[64]>(&x[0]));
        tmem_issue(aS + 64, *reinterpret_cast<uint32_t(*)[64]>(&x[64]));
        const uint4 gq = *const_cast<const uint4*>(&gone[seq % GONE]);
        const bool lost = (gq.x | gq.y | gq.z | gq.w) != 0;
        tmem_wait(*reinterpret_cast<uint32_t(*)[64]>(&x[0]));
        tmem_wait(*reinterpret_cast<uint32_t(*)[64]>(&x[64]));
        if (k0 + UBK > ctx || lost) {                    // nodes, the end, or a bad page
          const uint32_t g[4] = {gq.x, gq.y, gq.z, gq.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t bits = seen32(p, words, node, k0 + q * 32 - ctx) & ~g[q];
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((bits >> j) & 1u)) x[q * 32 + j] = 0xff800000u;
          }
        }
        float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
        for (int j = 0; j < 128; j += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mx[q] = fmax3(mx[q], __uint_as_float(x[j + 2 * q]), __uint_as_float(x[j + 2 * q + 1]));
        const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        // a new reference when the old one is more than 2^8 behind
        const bool move = mn > m && (m == neg_inf() || (mn - m) * c > 8.f);
        if (__any_sync(0xffffffffu, move && any)) {
          const float f = move && any ? (m == neg_inf() ? 0.f : ex2((m - mn) * c)) : 1.f;
          l *= f;
          // S(t) is out, so this stream's earlier products are complete
#pragma unroll
          for (int j = 0; j < DP / 16; ++j) {
            uint32_t o[16];
            tmem_issue(aO + j * 16, o);
            tmem_wait(o);
#pragma unroll
            for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
            tmem_store16(aO + j * 16, o);
          }
        }
        if (move) m = mn;
        const float ref = m == neg_inf() ? 0.f : m * c;
        float2 sum = make_float2(0.f, 0.f);
        const float2 c2 = make_float2(c, c), r2 = make_float2(-ref, -ref);
        // the weights become bf16 (off by at most 2^-8 each, the product's operand
        // type); the sum is that of the fp32 values
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t o[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 a = f2_fma(make_float2(__uint_as_float(x[q * 32 + 2 * j]),
                                                __uint_as_float(x[q * 32 + 2 * j + 1])), c2, r2);
            const float2 e = make_float2(ex2(a.x), ex2(a.y));
            sum = f2_add(sum, e);
            o[j] = pack2(e.x, e.y);
          }
          tmem_store16(aS + q * 16, o);
        }
        l += sum.x + sum.y;
        const int end = w.klen - k0;                     // tokens of the tile that exist
        if (end < UBK || lost) {
          // V rows that stand for no token: zero, so that 0 * V is 0
          const int pos = seq * 2 + 1, slot = pos % U::SLOTS;
          (void)wait(&full[slot], (uint32_t)(pos / U::SLOTS) & 1u);
          const uint32_t g[4] = {gq.x, gq.y, gq.z, gq.w};
          uint32_t mine = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if ((tl >> 5) == q) mine = g[q];
          if (tl >= end || ((mine >> (tl & 31)) & 1u)) {
            uint8_t* vr = ring + slot * U::SLOT + tl * 128;
#pragma unroll
            for (int hf = 0; hf < U::HALVES; ++hf)
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(vr + hf * (UBK * 128) + j * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tmem_store_wait();
        tc_fence_before();
        mbar_arrive(&pready[s]);
        any = true;
        ++done;
      }
      // the next item's queries, while the last product runs
      nx = w;
      more = nx.next(p, share);
      if (more) load_q(nx);
      if (any) {
        (void)wait(&pvdone[s], (uint32_t)(done - 1) & 1u);
        tc_fence_after();
      }
      const bool whole = w.t0 == 0 && w.t1 == w.nt;
      const int pslot = w.u == share.u0 ? 0 : 1;
      const int nd = valid ? node : 0;
      const long long o_row = ((long long)w.b * p.n + nd) * p.hq + w.h * p.g + (row - nd * p.g);
      const long long at = ((long long)blockIdx.x * 2 + pslot) * UBM + (w.split ? 0 : s * 128) + rr;
      const float ms = m == neg_inf() ? m : m * c;       // log2 units
      if (!w.split) {
        const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
        const float f = whole ? inv : 1.f;
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) {
          uint32_t o[16];
          tmem_issue(aO + j * 16, o);
          tmem_wait(o);
          if (!valid || j * 16 >= p.d) continue;
#pragma unroll
          for (int q = 0; q < 16; q += 8) {
            if (j * 16 + q >= p.d) continue;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(o[q + e]) * f;
            if (whole) {
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + o_row * p.d + j * 16 + q) =
                  make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
            } else {
              float4* d4 = reinterpret_cast<float4*>(p.po + at * p.d + j * 16 + q);
              d4[0] = make_float4(y[0], y[1], y[2], y[3]);
              d4[1] = make_float4(y[4], y[5], y[6], y[7]);
            }
          }
        }
        if (valid) {
          if (!whole) p.pml[at] = make_float2(ms, l);
          else if (p.lse) p.lse[o_row] = l > 0.f ? (ms + __log2f(l)) * kLn2 : (l == l ? neg_inf() : l);
        }
      } else {
        // the two streams hold the same rows: each group adds up half of the columns
        ml[s][rr] = make_float2(ms, any ? l : 0.f);
        tc_fence_before();
        pair_sync();
        tc_fence_after();
        const float2 a = ml[0][rr], b = ml[1][rr];
        const float mx = fmaxf(a.x, b.x), ref = mx == neg_inf() ? 0.f : mx;
        const float fa = ex2(a.x - ref), fb = ex2(b.x - ref);
        const bool two = w.t1 - w.t0 > 1;                // stream 1 had a tile
        const float sum = a.y * fa + (two ? b.y * fb : 0.f);
        const float inv = sum > 0.f ? 1.f / sum : (sum == sum ? 0.f : sum);
        const float f = whole ? inv : 1.f;
        const uint32_t a0 = tO + lane_base;
#pragma unroll
        for (int j2 = 0; j2 < DP / 32; ++j2) {
          const int j = s * (DP / 32) + j2;
          uint32_t o[16], o2[16];
          tmem_issue(a0 + j * 16, o);
          tmem_issue(a0 + DP + j * 16, o2);
          tmem_wait(o);
          tmem_wait(o2);
          if (!valid) continue;
#pragma unroll
          for (int q = 0; q < 16; q += 8) {
            if (j * 16 + q >= p.d) continue;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              y[e] = __uint_as_float(o[q + e]) * fa;
              if (two) y[e] = fmaf(__uint_as_float(o2[q + e]), fb, y[e]);
              y[e] *= f;
            }
            if (whole) {
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + o_row * p.d + j * 16 + q) =
                  make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
            } else {
              float4* d4 = reinterpret_cast<float4*>(p.po + at * p.d + j * 16 + q);
              d4[0] = make_float4(y[0], y[1], y[2], y[3]);
              d4[1] = make_float4(y[4], y[5], y[6], y[7]);
            }
          }
        }
        if (valid && s == 0) {
          if (!whole) p.pml[at] = make_float2(mx, sum);
          else if (p.lse) p.lse[o_row] = sum > 0.f ? (ref + __log2f(sum)) * kLn2 : (sum == sum ? neg_inf() : sum);
        }
        tc_fence_before();
        pair_sync();                                     // both accumulators are read
        tc_fence_after();
      }
      if (w.t0 == 0 && w.t1 < w.nt)
        begun = make_int4(w.b, w.h, w.mt, pslot | block_of(share, w.u + w.nt - 1) << 1);
      tc_fence_before();
    }
    if (warp == 2 && lane == 0) p.meta[blockIdx.x] = begun;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
  attn_tail<__nv_bfloat16>(p);
}

// [n_pages][heads][page places][d] as a 4D map; the place and the head in order of
// their strides. Boxes of 64 columns x min(page, 128) places.
bool encode_cache(CUtensorMap* map, const void* base, const AttnParams& p, int rows, int* slot_dim) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  // an axis of one entry is never stepped over: any valid stride will do
  const cuuint64_t row = (cuuint64_t)(p.d * 2 + 15) / 16 * 16;
  const cuuint64_t slot = p.page_size > 1 ? (cuuint64_t)p.ks_slot * 2 : row;
  const cuuint64_t head = p.hkv > 1 ? (cuuint64_t)p.ks_head * 2 : row;
  const cuuint64_t page = p.n_pages > 1 ? (cuuint64_t)p.ks_page * 2 : std::max(slot, head);
  *slot_dim = slot <= head ? 1 : 2;
  const bool one = *slot_dim == 1;
  const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)(one ? p.page_size : p.hkv),
                              (cuuint64_t)(one ? p.hkv : p.page_size), (cuuint64_t)p.n_pages};
  const cuuint64_t strides[3] = {one ? slot : head, one ? head : slot, page};
  const cuuint32_t box[4] = {64, one ? (cuuint32_t)rows : 1, one ? 1 : (cuuint32_t)rows, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i)
    if (strides[i] == 0 || strides[i] >= (1ull << 40)) return false;
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP>
cudaError_t run_umma(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v,
                     const UMaps& mp, int grid, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(attn_umma_kernel<DP>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)UShape<DP>::SMEM);
  if (e != cudaSuccess) return e;
  {
    TraceScope t(s, "attn_umma");
    attn_umma_kernel<DP><<<grid, UTHREADS, UShape<DP>::SMEM, s>>>(k, v, p, mp);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  TraceScope t(s, "attn_join");
  return launch_pdl(attn_join_kernel<__nv_bfloat16, UBM>, dim3(grid, UBM / 8), dim3(128), 0, s, 1, p);
}

}  // namespace

constexpr int kUmmaRows = UBM;
int attn_umma_rows() { return kUmmaRows; }

// Pages whose rows fill a swizzled tile without straddling it: a divisor of 128
// from 8 rows (the swizzle's period) up, or a multiple of 128.
bool attn_umma_pages(int page_size) {
  return page_size % 128 == 0 || (page_size >= 8 && 128 % page_size == 0);
}

// PCT_EUNSUPPORTED-like: cudaErrorNotSupported when the cache cannot be mapped.
cudaError_t launch_attn_umma(const AttnParams& p, int grid, cudaStream_t s) {
  CUtensorMap k, v;
  UMaps mp;
  mp.rows = p.page_size < 128 ? p.page_size : 128;
  mp.shift = 0;
  while ((1 << mp.shift) < mp.rows) ++mp.shift;
  if (!encode_cache(&k, p.k, p, mp.rows, &mp.slot_dim) ||
      !encode_cache(&v, p.v, p, mp.rows, &mp.slot_dim))
    return cudaErrorNotSupported;
  return p.d <= 64 ? run_umma<64>(p, k, v, mp, grid, s) : run_umma<128>(p, k, v, mp, grid, s);
}

}  // namespace pct
