// Tree attention for bf16 caches and many rows on the tcgen05 tensor cores.
//
// For calls of more than 32 rows (nodes x query heads of a group) a KV head: from some
// 64 on the two products outweigh the cache's bytes. One block an SM works on an item of two row tiles, R rows each
// (R = the largest multiple of the group up to 128), against key tiles of 64 tokens,
// as two streams:
//   * warp 0: TMA producer. Publishes the items, loads their queries (double
//     buffered) and streams K and V tiles through a ring of 128-byte swizzled
//     slots, a lane a box (a page's tokens in the tile, or 8, 16 or 32 of them);
//   * warps 1 and 2, one thread each: issue S = Q K^T (shared x shared) and O += P V
//     (P from tensor memory) of stream 0 and 1. A stream's scores are double
//     buffered, so its next S runs under the softmax of the current one. Two
//     issuers because issuing blocks while products run and each change between
//     the two kinds costs an issuer about 150 cycles: for a 64-token
//     tile of both streams one thread takes 1768 cycles, two threads 1269;
//   * warps 3-6 and 7-10: the softmax of stream 0 and 1. A thread reads its row of
//     64 scores from tensor memory, keeps the running maximum and sum, and writes
//     the weights back as bf16 over the scores. At an item's end they leave the
//     rows in the item's query buffer;
//   * warp 11: stores these rows by TMA (boxes like the queries'; rows past count
//     are staged as zeros) and hands the buffer back to the producer. With the
//     softmax warps storing them an item cost as much as 5.6 tiles.
// (head_dim above 128: one stream and one row tile, whose accumulator takes half of
// tensor memory.) With more than R rows in an item the streams are its two row tiles and share
// every K and V tile; with fewer they take alternate key tiles of the same rows
// and are added up at the item's end (both accumulators sit in the same tensor
// memory lanes). Tensor memory: S (2 streams x 2 buffers x 64 columns, P in the
// first 32 of its S), then O_0, O_1. The accumulator is rescaled only when a row's
// maximum grows by more than 2^8 over the one in use, which the later tiles seldom do;
// weights are taken relative to 2^8 times that one, so none is above 1.
// 64 tokens a tile rather than 128: with 128 the scores fill tensor memory once
// (head_dim 128), so that S, softmax and P V of a stream run one after another
// (64 requests x 256 nodes over up to 4096 tokens: 1.41 ms; this takes 0.75-0.93,
// 600-740 TFLOP/s, by the clock that the power limit leaves). A 64-token tile of both streams takes about 2000 cycles, 1270 of
// products alone and 1024 of exponentials, which overlap in part.
// Every mbarrier wait is bounded; when one gives up, the roles run to the end
// without waiting, drain their copies and products, free the tensor memory, and
// the join reports PCT_DEV_TIMEOUT.
#include <cuda.h>

#include <algorithm>

#include "attn_sched.cuh"
#include "umma.cuh"

namespace pct {
namespace {

constexpr int UBK = 64;                  // tokens of a key tile
constexpr int UTHREADS = 384;
constexpr int UROWS = 256;               // row places of a piece (two streams of 128)
constexpr int GONE = 8;                  // tiles whose bad-page marks are kept
constexpr int ITEMS = 8;                 // published items

template <int DP> struct UShape {
  static constexpr int STREAMS = DP == 256 ? 1 : 2;        // (two accumulators fill tensor memory)
  static constexpr int HALVES = DP / 64;                   // 64-column boxes of a row
  static constexpr int QHALF = 128 * 128;                  // bytes of 128 rows of a box
  static constexpr int QTILE = HALVES * QHALF;
  static constexpr int KHALF = UBK * 128;
  static constexpr int SLOT = HALVES * KHALF;
  static constexpr int SLOTS = DP == 256 ? 3 : DP == 128 ? 6 : 8;   // K and V tiles in flight
  static constexpr size_t SMEM = 1024 + 2 * STREAMS * QTILE + SLOTS * SLOT;
};

struct UMaps {
  int shift;                             // log2 of a box's tokens
  int slot_dim;                          // cache map axis of the token in a page: 1 or 2
  int rows;                              // R
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int x, int y,
                                             int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z), "r"(w), "r"(src)
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
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// An item as the producer publishes it. seq numbers the key tiles that the block
// loads (their ring slots follow from it). The producer publishes item i only when
// both softmax groups are done with item i - 2 (their query buffers are free), and
// loads no tile further than the ring's SLOTS / 2 past one that an issuer has not
// handed back. An item has a tile at least, and each issuer passes every tile of it, so
// no entry of ITEMS is written while a role still has to read it.
struct Item {
  int b, h, mt, t0, t1, rows, klen, ctx, seq;
  int last;                              // no more items; the rest is not set
  int split;                             // streams on alternate tiles of the same rows
  int whole, pslot;                      // written out directly, or the piece's slot
  __device__ int start(int st) const { return split ? t0 + st : t0; }
  __device__ int step() const { return split ? 2 : 1; }
};

// The factor from scores to exponents of a row with maximum m: c, but for |m c| from 2^28 on
// (infinities too) the power of two that brings |m| into [2^30, 2^31). A weight is
// 2^(x c - ref) with ref = m c rounded once, so the maximum's own is off by half a step of ref
// in the exponent: at most 8 below 2^28, past an exponential's range from 2^31 on. With a power
// of two it is exact. There two scores next to each other differ by 2^4 at least with c and by
// 2^6 at least with the power of two: the maximum's weight is 1 and any smaller score's nothing.
__device__ __forceinline__ float row_factor(float m, float c) {
  if (!(fabsf(m) * c >= 268435456.f) || m == neg_inf()) return c;
  const uint32_t e = (__float_as_uint(m) >> 23) & 255u;
  return __uint_as_float(min(284u - e, 254u) << 23);
}

// The reference of a row's weights: 8 above its m, which may be that far behind the running
// maximum, so that no weight is above 1 and large values overflow no sooner than with the
// maximum itself. (With row_factor's power of two m is never behind.)
__device__ __forceinline__ float row_ref(float m, float cr, float c) {
  return fmaf(m, cr, cr == c ? 8.f : 0.f);
}

// One accumulator column pair of 8: 16 bytes of a bf16 row.
__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  return make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
}

template <int DP>
__global__ void __launch_bounds__(UTHREADS, 1)
attn_umma_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                 const AttnParams p, const UMaps mp) {
  typedef UShape<DP> U;
  constexpr int STREAMS = U::STREAMS;
  static_assert(U::SLOTS / 2 < ITEMS && U::SLOTS / 2 < GONE, "entries outlive the ring's tiles");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));   // [stream][2]
  uint8_t* ring = sQ + 2 * STREAMS * U::QTILE;
  __shared__ uint64_t full[U::SLOTS], empty[U::SLOTS], qfull[2][2], qempty[2][2], sfull[2][2],
      pready[2][2], pvdone[2][2], staged[2][2], item_full[ITEMS], pair, drain[2];
  __shared__ Item items[ITEMS];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ uint2 gone[GONE];
  __shared__ Share share;
  __shared__ long long sums[UTHREADS / 32];
  volatile int* abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* err = p.fail + blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < U::SLOTS; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], STREAMS); }
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < 2; ++j) {
        mbar_init(&qfull[i][j], 1);
        mbar_init(&qempty[i][j], 1);
        mbar_init(&staged[i][j], 128);
        mbar_init(&sfull[i][j], 1);
        mbar_init(&pready[i][j], 128);
        mbar_init(&pvdone[i][j], 1);
      }
      mbar_init(&drain[i], 1);
    }
    for (int i = 0; i < ITEMS; ++i) mbar_init(&item_full[i], 1);
    mbar_init(&pair, 256);
    abort_word = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_slot)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();      // the set-up above touches only shared memory and TMEM
  pdl_trigger();
  if (tid == 0) *err = 0;
  sched_begin<UBK, UTHREADS>(p, &share, sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = tmem_slot, tO = tS + 256;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    Walk<UBK> w;
    w.begin(share);
    int seq0 = 0, n_items = 0;
    int4 begun = make_int4(-1, 0, 0, 0);
    bool ok = true;
    uint32_t armed = 0;                              // ring slots used
    bool lost_page = false;
    int slot = 0;
    uint32_t par = 0;
    const int boxes = UBK >> mp.shift;               // boxes of a tile
    const int nodes = mp.rows / p.g;                 // nodes of a row tile
    while (ok) {
      const bool end = !w.next(p, share, &begun);
      const int b = w.b, h = w.h, mt = w.mt - 1, t0 = w.t0, t1 = w.t1, klen = w.klen, rows = w.rows;
      const int buf = n_items & 1;
      const uint32_t qpar = (uint32_t)(n_items >> 1) & 1u;
#pragma unroll
      for (int s = 0; s < STREAMS; ++s) {
        // the buffer's reader is done, and so is the copy before (a stream without
        // tiles does not wait for its queries)
        bool got = wait_bar(&qempty[s][buf], qpar ^ 1u, abort_flag, err);
        if (n_items >= 2) got = got && wait_bar(&qfull[s][buf], qpar ^ 1u, abort_flag, err);
        if (!__all_sync(0xffffffffu, got)) ok = false;
      }
      if (!ok) break;
      const bool split = STREAMS == 2 && rows <= mp.rows;
      if (lane == 0) {
        Item& it = items[n_items % ITEMS];
        it.b = b; it.h = h; it.mt = mt; it.t0 = t0; it.t1 = t1; it.rows = rows; it.klen = klen;
        it.ctx = (int)w.r.ctx; it.seq = seq0; it.last = end; it.split = split;
        it.whole = w.whole;
        it.pslot = w.pslot;
        mbar_arrive(&item_full[n_items % ITEMS]);
        if (!end) {
#pragma unroll
          for (int s = 0; s < STREAMS; ++s) {
            mbar_expect_tx(&qfull[s][buf], (uint32_t)(mp.rows * 128 * U::HALVES));
            const int node = (mt * STREAMS + (split ? 0 : s)) * nodes;
            const uint32_t dst = smem_u32(sQ + (s * 2 + buf) * U::QTILE);
#pragma unroll
            for (int hf = 0; hf < U::HALVES; ++hf)
              tma_load_4d(dst + hf * U::QHALF, &tmQ, hf * 64, h * p.g, node, b, &qfull[s][buf]);
          }
        }
      }
      __syncwarp();
      if (end) break;
      ++n_items;
      const int32_t* table = p.table + (long long)b * p.max_pages;
      for (int t = t0; t < t1 && ok; ++t) {
        const int seq = seq0 + t - t0;
        const int tok = t * UBK + (lane << mp.shift);
        int page = -1, place = 0;
        const bool live = lane < boxes && tok < klen;
        if (live) {
          const uint32_t col = page_of(p, tok);
          page = __ldg(table + col);
          place = tok - (int)col * p.page_size;
          if (page >= p.n_pages) page = -1;
        }
        const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
        const uint32_t lost = __ballot_sync(0xffffffffu, live && page < 0);
        lost_page |= lost != 0;
        if (lane == 0) {
          uint32_t g[2] = {0, 0};
          for (int i = 0; lost >> i; ++i)
            if ((lost >> i) & 1)
              for (int k = i << mp.shift; k < (i + 1) << mp.shift; ++k) g[k >> 5] |= 1u << (k & 31);
          gone[seq % GONE] = make_uint2(g[0], g[1]);
        }
        const uint32_t bytes = (uint32_t)__popc(have) * (128u << mp.shift) * U::HALVES;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const bool got = wait_bar(&empty[slot], par ^ 1u, abort_flag, err);
          if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
          if (lane == 0) mbar_expect_tx(&full[slot], bytes);
          __syncwarp();
          if (page >= 0) {
            const uint32_t dst = smem_u32(ring + slot * U::SLOT) + ((uint32_t)lane << mp.shift) * 128u;
            const int y = mp.slot_dim == 1 ? place : h, z = mp.slot_dim == 1 ? h : place;
#pragma unroll
            for (int hf = 0; hf < U::HALVES; ++hf)
              tma_load_4d(dst + hf * U::KHALF, kv ? &tmV : &tmK, hf * 64, y, z, page, &full[slot]);
          }
          armed |= 1u << slot;
          if (++slot == U::SLOTS) { slot = 0; par ^= 1u; }
        }
      }
      seq0 += t1 - t0;
    }
    if (lane == 0) {
      p.meta[blockIdx.x] = begun;
      if (lost_page) atomicOr(err, FAIL_PAGE);
    }
    // every copy has landed before the block may exit: slot i was last armed in the
    // current round when i < slot, in the one before otherwise
#pragma unroll
    for (int i = 0; i < U::SLOTS; ++i)
      if (armed & (1u << i)) drain_wait(&full[i], i < slot ? par : par ^ 1u);
    for (int i = max(0, n_items - 2); i < n_items; ++i)
      for (int s = 0; s < STREAMS; ++s) drain_wait(&qfull[s][i & 1], (uint32_t)(i >> 1) & 1u);
  } else if (warp <= 2) {
    if (lane == 0 && warp <= STREAMS) {
      // ---------------- products of stream s ----------------
      constexpr uint32_t BASE = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 4) << 24);
      constexpr uint32_t ID_QK = BASE | ((uint32_t)(UBK >> 3) << 17);
      constexpr uint32_t ID_PV = BASE | (1u << 16) | ((uint32_t)(DP >> 3) << 17);
      const int s = warp - 1;
      const uint64_t q_desc = make_desc(smem_u32(sQ + s * 2 * U::QTILE), 16, 1024);
      const uint64_t k_desc = make_desc(smem_u32(ring), 16, 1024);
      const uint64_t v_desc = make_desc(smem_u32(ring), U::KHALF, 1024);
      // Every issuer waits for every fill of every ring slot and hands it back, also
      // for the other stream's tiles of a split item: a parity tells a fill from the one
      // before only to a reader that has seen the one before arrive.
      // The item in hand, its next tile and its end, the first of this stream; S and
      // P V issued
      int item = -1, t = 0, t1 = 0, mine = 0, seq = 0, step = 1, n_s = 0, n_pv = 0;
      // per score buffer, of the P V to come: V's ring position << 1 | first
      int todo0 = 0, todo1 = 0;
      bool head = true, live = true;
      long long c0 = 0;
      uint32_t spins = 0;
      while (live || n_pv < n_s) {
        // the P V of the older tile where its weights are there, else the next S;
        // neither waits for the other (the next item may need this P V)
        bool moved = false;
        if (n_pv < n_s) {
          const int bf = n_pv & 1, td = bf ? todo1 : todo0;
          const int pos = td >> 1, slot = pos % U::SLOTS;
          if (mbar_test(&pready[s][bf], (uint32_t)(n_pv >> 1) & 1u) &&
              mbar_test(&full[slot], (uint32_t)(pos / U::SLOTS) & 1u)) {
            tc_fence_after();
            const uint64_t vd = v_desc + (uint64_t)((slot * U::SLOT) >> 4);
            const uint32_t more = !(td & 1);
#pragma unroll
            for (int k = 0; k < UBK / 16; ++k)
              umma_ts(tO + s * DP, tS + s * 128 + bf * 64 + k * 8, vd + (uint64_t)((k * 2048) >> 4),
                      ID_PV, more | (k > 0));
            umma_commit(&pvdone[s][bf]);
            umma_commit(&empty[slot]);
            ++n_pv;
            moved = true;
          }
        }
        if (live && t >= t1) {                          // the next item
          const int i = item + 1;
          if (mbar_test(&item_full[i % ITEMS], (uint32_t)(i / ITEMS) & 1u)) {
            const Item& it = items[i % ITEMS];
            item = i;
            if (it.last) {
              live = false;
            } else {
              t = it.t0;
              t1 = it.t1;
              mine = it.start(s);
              step = it.step();
              seq = it.seq - it.t0;
              head = true;
            }
            moved = true;
          }
        } else if (live && step == 2 && ((t ^ mine) & 1)) {   // the other stream's tile
          const int pos = (seq + t) * 2, ks = pos % U::SLOTS, vs = (pos + 1) % U::SLOTS;
          // (of a V tile that this stream has still to multiply, the slot's next fill
          // cannot be told yet)
          const bool seen = n_pv == n_s || (((n_pv & 1) ? todo1 : todo0) >> 1) + U::SLOTS > pos + 1;
          if (seen && mbar_test(&full[ks], (uint32_t)(pos / U::SLOTS) & 1u) &&
              mbar_test(&full[vs], (uint32_t)((pos + 1) / U::SLOTS) & 1u)) {
            mbar_arrive(&empty[ks]);
            mbar_arrive(&empty[vs]);
            ++t;
            moved = true;
          }
        } else if (live && n_s - n_pv < 2) {
          const int bf = n_s & 1, pos = (seq + t) * 2, slot = pos % U::SLOTS;
          if (mbar_test(&full[slot], (uint32_t)(pos / U::SLOTS) & 1u) &&
              (n_s < 2 || mbar_test(&pvdone[s][bf], (uint32_t)((n_s >> 1) - 1) & 1u)) &&
              mbar_test(&qfull[s][item & 1], (uint32_t)(item >> 1) & 1u)) {
            tc_fence_after();
            const uint64_t qd = q_desc + (uint64_t)(((item & 1) * U::QTILE) >> 4);
            const uint64_t kd = k_desc + (uint64_t)((slot * U::SLOT) >> 4);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
              umma_f16(tS + s * 128 + bf * 64,
                       qd + (uint64_t)(((k >> 2) * U::QHALF + (k & 3) * 32) >> 4),
                       kd + (uint64_t)(((k >> 2) * U::KHALF + (k & 3) * 32) >> 4), ID_QK, k > 0);
            umma_commit(&sfull[s][bf]);
            umma_commit(&empty[slot]);
            const int td = (pos + 1) << 1 | (head ? 1 : 0);
            if (bf) todo1 = td; else todo0 = td;
            ++n_s;
            head = false;
            ++t;
            moved = true;
          }
        }
        if (moved) {
          spins = 0;
        } else if ((++spins & 255u) == 0u) {
          if (spins == 256u) c0 = clock64();
          if (*abort_flag) break;
          if (clock64() - c0 > kTimeoutCycles) {
            *abort_flag = 1;
            atomicOr(err, FAIL_TIMEOUT);
            break;
          }
        }
      }
      umma_commit(&drain[s]);
      drain_wait(&drain[s], 0);
    }
  } else if (warp == 11) {
    if (lane == 0) {
      // ---------------- output rows ----------------
      const int nodes = mp.rows / p.g;
      for (int i = 0;; ++i) {
        if (!wait_bar(&item_full[i % ITEMS], (uint32_t)(i / ITEMS) & 1u, abort_flag, err)) break;
        const Item& w = items[i % ITEMS];
        if (w.last) break;
        const int buf = i & 1;
        const uint32_t par = (uint32_t)(i >> 1) & 1u;
        bool got = true;
#pragma unroll
        for (int s = 0; s < STREAMS; ++s) {
          got = got && wait_bar(&staged[s][buf], par, abort_flag, err);
          // both streams of a split item stage in stream 0's buffer
          const int first = (w.mt * STREAMS + s) * nodes;
          if (got && w.whole && (w.split ? s == 1 : first < p.n)) {
            const uint32_t src = smem_u32(sQ + ((w.split ? 0 : s) * 2 + buf) * U::QTILE);
#pragma unroll
            for (int hf = 0; hf < U::HALVES; ++hf)
              if (hf * 64 < p.d) tma_store_4d(&tmO, src + hf * U::QHALF, hf * 64, w.h * p.g,
                           w.split ? w.mt * 2 * nodes : first, w.b);
          }
        }
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        if (!got) break;                                 // (the group so far is waited for below)
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
#pragma unroll
        for (int s = 0; s < STREAMS; ++s) mbar_arrive(&qempty[s][buf]);
      }
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
  } else {
    // ---------------- softmax ----------------
    const int s = (warp - 3) >> 2, quad = warp & 3;
    const int tl = quad * 32 + lane;                     // thread of the group, row of the
                                                         // stream, tensor memory lane
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint32_t aS = tS + s * 128 + lane_base, aO = tO + s * DP + lane_base;
    const float c = p.scale_log2;
    int n = 0, n_items = 0;                              // tiles of this stream, items
    attn_zero<__nv_bfloat16>(p, s * 128 + tl, 256);      // while the first tiles arrive
    uint32_t met = 0;
    auto wait = [&](uint64_t* bar, uint32_t par) {
      const bool got = wait_bar(bar, par, abort_flag, err);
      return __all_sync(0xffffffffu, got);
    };
    auto pair_sync = [&]() {                             // both softmax groups (bounded)
      mbar_arrive(&pair);
      (void)wait(&pair, met++ & 1u);
    };
    for (; s < STREAMS; ++n_items) {
      const int slot_i = n_items % ITEMS, buf = n_items & 1;
      if (!wait(&item_full[slot_i], (uint32_t)(n_items / ITEMS) & 1u)) break;
      const Item& w = items[slot_i];
      if (w.last) break;
      const bool split = w.split, whole = w.whole;
      const int off = split ? 0 : s * mp.rows;           // the stream's first row of the item
      const int lim = min(mp.rows, w.rows - off);
      const int row0 = w.mt * p.bm + off;
      const bool valid = tl < lim;
      const int node = valid ? (row0 + tl) / p.g : -0x40000000;
      const uint32_t* words =
          p.mask && valid ? p.mask + ((long long)w.b * p.n + node) * p.words : nullptr;
      const int ctx = w.ctx, seq0 = w.seq - w.t0, klen = w.klen, t1 = w.t1, step = w.step();
      float m = neg_inf(), l = 0.f, cr = c, ref = 0.f;
      const int n0 = n;
      for (int t = w.start(s); t < t1; t += step, ++n) {
        const int seq = seq0 + t, k0 = t * UBK, bf = n & 1;
        (void)wait(&sfull[s][bf], (uint32_t)(n >> 1) & 1u);
        tc_fence_after();
        uint32_t x[64];
        __syncwarp();
        tmem_issue(aS + bf * 64, x);
        const uint2 gq = *const_cast<const uint2*>(&gone[seq % GONE]);
        const bool lost = (gq.x | gq.y) != 0;
        tmem_wait(x);
        if (k0 + UBK > ctx || lost) {                    // nodes, the end, or a bad page
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t bits = seen32(p, words, node, k0 + q * 32 - ctx) & ~(q ? gq.y : gq.x);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((bits >> j) & 1u)) x[q * 32 + j] = 0xff800000u;
          }
        }
        float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
        for (int j = 0; j < 64; j += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mx[q] = fmax3(mx[q], __uint_as_float(x[j + 2 * q]), __uint_as_float(x[j + 2 * q + 1]));
        const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        // a new reference when the old one is more than 2^8 behind
        const bool move = valid && mn > m && (m == neg_inf() || (mn - m) * c > 8.f);
        if (n > n0 && __any_sync(0xffffffffu, move)) {
          const float f = move ? (m == neg_inf() ? 0.f : ex2((m - mn) * c)) : 1.f;
          l *= f;
          // every product of this stream before P V of this tile is complete
          (void)wait(&pvdone[s][bf ^ 1], (uint32_t)((n - 1) >> 1) & 1u);
          tc_fence_after();
          __syncwarp();
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
        if (move) {
          m = mn;
          cr = row_factor(m, c);
          ref = row_ref(m, cr, c);
        }
        float2 sum = make_float2(0.f, 0.f);
        const float2 c2 = make_float2(cr, cr), r2 = make_float2(-ref, -ref);
        __syncwarp();                                    // the stores take a converged warp
        // the weights become bf16 (off by at most 2^-8 each, the product's operand
        // type); the sum is that of the fp32 values
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t o[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 a = f2_fma(make_float2(__uint_as_float(x[q * 32 + 2 * j]),
                                                __uint_as_float(x[q * 32 + 2 * j + 1])), c2, r2);
            const float2 e = make_float2(ex2(a.x), ex2(a.y));
            sum = f2_add(sum, e);
            o[j] = pack2(e.x, e.y);
          }
          tmem_store16(aS + bf * 64 + q * 16, o);
        }
        l += sum.x + sum.y;
        const int end = klen - k0;                       // tokens of the tile that exist
        if (end < UBK || lost) {
          // V rows that stand for no token: zero, so that 0 * V is 0. (The fill before
          // this one in the slot has arrived: it was multiplied at the latest with
          // this stream's tile before, or handed back before this tile's S.)
          if (n > 0) (void)wait(&pvdone[s][bf ^ 1], (uint32_t)((n - 1) >> 1) & 1u);
          const int pos = seq * 2 + 1, slot = pos % U::SLOTS;
          (void)wait(&full[slot], (uint32_t)(pos / U::SLOTS) & 1u);
          if (tl < UBK && (tl >= end || (((tl < 32 ? gq.x : gq.y) >> (tl & 31)) & 1u))) {
            uint8_t* vr = ring + slot * U::SLOT + tl * 128;
#pragma unroll
            for (int hf = 0; hf < U::HALVES; ++hf)
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(vr + hf * U::KHALF + j * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
        }
        __syncwarp();
        tmem_store_wait();
        tc_fence_before();
        mbar_arrive(&pready[s][bf]);
      }
      const bool any = n > n0;
      if (any) {
        (void)wait(&pvdone[s][(n - 1) & 1], (uint32_t)((n - 1) >> 1) & 1u);
        tc_fence_after();
      }
      // O to the caller, through this item's query buffer (its products are complete);
      // pieces directly, [d / 4][row][4]
      const float ms = m == neg_inf() ? m : row_ref(m, c, c);   // log2 units
      const long long piece = (long long)blockIdx.x * 2 + w.pslot;
      const int place = (split ? 0 : s * 128) + tl;
      float4* po = reinterpret_cast<float4*>(p.po) + piece * (p.d / 4) * UROWS + place;
      uint8_t* stage = sQ + ((split ? 0 : s) * 2 + buf) * U::QTILE + tl * 128;
      auto put = [&](int col, const float (&y)[8]) {     // 8 columns from `col`
        if (whole) {
          const int ch = col / 8;
          *reinterpret_cast<uint4*>(stage + (ch >> 3) * U::QHALF + (((ch & 7) ^ (tl & 7)) << 4)) =
              valid ? pack8(y) : make_uint4(0, 0, 0, 0);
        } else if (valid && col < p.d) {
          po[(col / 4) * UROWS] = make_float4(y[0], y[1], y[2], y[3]);
          po[(col / 4 + 1) * UROWS] = make_float4(y[4], y[5], y[6], y[7]);
        }
      };
      // (a stream without tiles has not seen its queries arrive)
      (void)wait(&qfull[s][buf], (uint32_t)(n_items >> 1) & 1u);
      float row_m = ms, row_l = l;
      if (STREAMS == 1 || !split) {
        const float f = whole ? inverse(l) : 1.f;
#pragma unroll
        for (int j = 0; j < DP / 64; ++j) {
          uint32_t o[64];
          __syncwarp();
          tmem_issue(aO + j * 64, o);
          tmem_wait(o);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(o[q * 8 + e]) * f;
            put(j * 64 + q * 8, y);
          }
        }
      } else {
        // the two streams hold the same rows: each group adds up half of the columns
        // (maxima and sums meet in stream 1's query buffer, free once both are here)
        const int col0 = s * (DP / 2);
        float2* ml = reinterpret_cast<float2*>(sQ + (2 + buf) * U::QTILE) + tl;
        tc_fence_before();
        pair_sync();
        tc_fence_after();
        ml[s * 128] = make_float2(ms, l);
        pair_sync();
        const float2 a = ml[0], b = ml[128];
        row_m = fmaxf(a.x, b.x);
        const float ref = row_m == neg_inf() ? 0.f : row_m;
        const float fa = ex2(a.x - ref), fb = ex2(b.x - ref);
        const bool two = t1 - w.t0 > 1;                  // stream 1 had a tile
        row_l = a.y * fa + b.y * fb;
        const float f = whole ? inverse(row_l) : 1.f;
        const uint32_t a0 = tO + lane_base + col0;
#pragma unroll
        for (int j = 0; j < DP / 64; ++j) {
          uint32_t o[32], o2[32];
          __syncwarp();
          tmem_issue(a0 + j * 32, o);
          tmem_issue(a0 + DP + j * 32, o2);
          tmem_wait(o);
          tmem_wait(o2);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              y[e] = __uint_as_float(o[q * 8 + e]) * fa;
              if (two) y[e] = fmaf(__uint_as_float(o2[q * 8 + e]), fb, y[e]);
              y[e] *= f;
            }
            put(col0 + j * 32 + q * 8, y);
          }
        }
        tc_fence_before();
        pair_sync();                                     // both accumulators are read
        tc_fence_after();
      }
      if (valid && !(split && s == 1)) {
        if (!whole) p.pml[piece * UROWS + place] = make_float2(row_m, row_l);
        else if (p.lse)
          p.lse[((long long)w.b * p.n + node) * p.hq + w.h * p.g + (row0 + tl - node * p.g)] =
              lse_of(row_m == neg_inf() ? 0.f : row_m, row_l);
      }
      fence_async_smem();                                // the buffer's next user is a copy
      tc_fence_before();
      mbar_arrive(&staged[s][buf]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tS), "r"(512));
  }
}

// Joins the pieces of the split item that block blockIdx.x began: a thread a row and
// NC 4-column groups, 16 apart (blockIdx.y: 8 groups of 32 rows x 4 of columns; one request of 64
// nodes over 8000 tokens takes 46, 41, 37 and 42 us with 1, 2, 4 and 8 of columns).
template <int NC>
__global__ void __launch_bounds__(128) attn_umma_join_kernel(AttnParams p, int rows_tile) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x;
  const int4 m = p.meta[c];
  if (blockIdx.y == 0) attn_status(p);
  if (m.x < 0) return;
  const int b = m.x, h = m.y & 1023, rows = m.y >> 10, mt = m.z, slot = m.w & 1, last = m.w >> 1;
  const int place = (blockIdx.y >> 2) * 32 + (threadIdx.x & 31);
  const int w = (blockIdx.y & 3) * 4 + (threadIdx.x >> 5);       // column groups w, w + 16, ..
  const int s = place >> 7, rr = place & 127;
  const int d4 = p.d / 4;
  if (rr >= rows_tile || s * rows_tile + rr >= rows || w >= d4) return;
  JoinState st;
  st.begin();
  float4 acc[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int AHEAD = JOIN_AHEAD * 2 / NC;
  for (int k0 = c; k0 <= last; k0 += AHEAD) {
    float2 a[AHEAD];
    float4 x[AHEAD][NC];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int k = min(k0 + j, last);
      const long long at = (long long)k * 2 + (k == c ? slot : 0);
      const float4* po = reinterpret_cast<const float4*>(p.po) + at * d4 * UROWS + place;
      a[j] = p.pml[at * UROWS + place];
#pragma unroll
      for (int i = 0; i < NC; ++i) x[j][i] = po[(w + 16 * i < d4 ? w + 16 * i : w) * UROWS];
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (k0 + j > last) break;
      const float2 f = st.add(a[j]);
#pragma unroll
      for (int i = 0; i < NC; ++i) join_add(acc[i], x[j][i], f);
    }
  }
  const int row = mt * p.bm + s * rows_tile + rr, node = row / p.g;
  const long long o = ((long long)b * p.n + node) * p.hq + h * p.g + (row - node * p.g);
  const float inv = inverse(st.l);
#pragma unroll
  for (int j = 0; j < NC; ++j)
    if (w + 16 * j < d4)
      store_out(static_cast<__nv_bfloat16*>(p.out) + o * p.d + (w + 16 * j) * 4,
                make_float4(acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv));
  if (p.lse && w == 0) p.lse[o] = lse_of(st.m == neg_inf() ? 0.f : st.m, st.l);
}

bool encode_4d(CUtensorMap* map, const void* base, const cuuint64_t (&dims)[4],
               const cuuint64_t (&strides)[3], const cuuint32_t (&box)[4]) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  for (int i = 0; i < 3; ++i)
    if (strides[i] == 0 || strides[i] >= (1ull << 40)) return false;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// [n_pages][heads][page places][d]; the place and the head in order of their strides.
// Boxes of 64 columns x `rows` places. (An axis of one entry is never
// stepped over: any valid stride will do for it.)
bool encode_cache(CUtensorMap* map, const void* base, const AttnParams& p, int rows, int* slot_dim) {
  const cuuint64_t row = (cuuint64_t)(p.d * 2 + 15) / 16 * 16;
  const cuuint64_t slot = p.page_size > 1 ? (cuuint64_t)p.ks_slot * 2 : row;
  const cuuint64_t head = p.hkv > 1 ? (cuuint64_t)p.ks_head * 2 : row;
  const cuuint64_t page = p.n_pages > 1 ? (cuuint64_t)p.ks_page * 2 : std::max(slot, head);
  const bool one = slot <= head;
  *slot_dim = one ? 1 : 2;
  const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)(one ? p.page_size : p.hkv),
                              (cuuint64_t)(one ? p.hkv : p.page_size), (cuuint64_t)p.n_pages};
  const cuuint64_t strides[3] = {one ? slot : head, one ? head : slot, page};
  const cuuint32_t box[4] = {64, one ? (cuuint32_t)rows : 1, one ? 1 : (cuuint32_t)rows, 1};
  return encode_4d(map, base, dims, strides, box);
}
// [batch][n][heads][d], boxes of 64 columns x a group's heads x the nodes of a row tile
bool encode_rows(CUtensorMap* map, const void* base, const AttnParams& p, int64_t s_b, int64_t s_n,
                 int64_t s_h, int nodes) {
  const cuuint64_t row = (cuuint64_t)(p.d * 2 + 15) / 16 * 16;
  const cuuint64_t head = p.hq > 1 ? (cuuint64_t)s_h * 2 : row;
  const cuuint64_t node = p.n > 1 ? (cuuint64_t)s_n * 2 : head;
  const cuuint64_t req = p.batch > 1 ? (cuuint64_t)s_b * 2 : node;
  const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.hq, (cuuint64_t)p.n, (cuuint64_t)p.batch};
  const cuuint64_t strides[3] = {head, node, req};
  const cuuint32_t box[4] = {64, (cuuint32_t)p.g, (cuuint32_t)nodes, 1};
  return encode_4d(map, base, dims, strides, box);
}

template <int DP>
cudaError_t run_umma(const AttnParams& p, const CUtensorMap& q, const CUtensorMap& k,
                     const CUtensorMap& v, const CUtensorMap& o, const UMaps& mp, int grid,
                     cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(attn_umma_kernel<DP>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)UShape<DP>::SMEM);
  if (e != cudaSuccess) return e;
  {
    TraceScope t(s, "attn_umma");
    e = launch_pdl(attn_umma_kernel<DP>, dim3(grid), dim3(UTHREADS), UShape<DP>::SMEM, s, 1, q, k,
                   v, o, p, mp);
  }
  if (e != cudaSuccess) return e;
  TraceScope t(s, "attn_umma_join");
  return launch_pdl(attn_umma_join_kernel<DP == 256 ? 4 : 2>, dim3(grid, UROWS / 32 * 4), dim3(128), 0, s, 1, p, mp.rows);
}

}  // namespace

int attn_umma_rows() { return UROWS; }

// A box holds the largest power of two of tokens that divides the page, at most a
// tile: it never straddles a page, and from 8 rows on (the swizzle's period) it keeps
// the tile's layout.
int box_rows(int page_size) { return std::min(page_size & -page_size, UBK); }
bool attn_umma_pages(int page_size) { return box_rows(page_size) >= 8; }

// cudaErrorNotSupported when the strides do not fit a tensor map.
cudaError_t launch_attn_umma(AttnParams p, int grid, cudaStream_t s) {
  CUtensorMap q, k, v, o;
  UMaps mp;
  const int rows = box_rows(p.page_size);
  mp.shift = 0;
  while ((1 << mp.shift) < rows) ++mp.shift;
  const int nodes = 128 / p.g;
  mp.rows = nodes * p.g;
  p.bm = (p.d > 128 ? 1 : 2) * mp.rows;
  // costs fitted to the cycles of 148 blocks over mixed items
  p.half = mp.rows;
  p.many = 4;
  p.few = 3;
  p.per_item = 8;
  const int64_t row = (int64_t)p.hq * p.d;
  if (!encode_rows(&q, p.q, p, p.qs_b, p.qs_n, p.qs_h, nodes) ||
      !encode_rows(&o, p.out, p, row * p.n, row, p.d, nodes) || !encode_cache(&k, p.k, p, rows, &mp.slot_dim) ||
      !encode_cache(&v, p.v, p, rows, &mp.slot_dim))
    return cudaErrorNotSupported;
  if (p.d <= 64) return run_umma<64>(p, q, k, v, o, mp, grid, s);
  if (p.d <= 128) return run_umma<128>(p, q, k, v, o, mp, grid, s);
  return run_umma<256>(p, q, k, v, o, mp, grid, s);
}

}  // namespace pct
