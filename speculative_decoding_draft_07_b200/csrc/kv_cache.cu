// The paged cache's bookkeeping and data movement: block tables from lengths
// (kv_pages_resize), slots and positions (kv_tree_slots), new rows into their
// slots (kv_append) and the accepted path's rows behind the context (kv_commit).
// None computes anything: the first two are bound by latency (one launch, few
// dependent reads), the last two by the bytes that move (16 bytes a thread, the
// loads of a thread issued before its stores).
#include "common.cuh"
#include "internal.h"

namespace pct {
namespace {

constexpr int kResizeThreads = 1024;

// Exclusive scan of one value per thread over the block; returns the prefix and
// the total. The first barrier lets a previous call's readers finish.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums,
                                                long long* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[w] = inc;
  __syncthreads();
  if (w == 0) {
    long long s = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[(blockDim.x >> 5) - 1];
  const long long base = w > 0 ? warp_sums[w - 1] : 0;
  return base + inc - x;
}

// One block: the requests in chunks of blockDim, and within a chunk the pages
// that move spread evenly over the threads (each finds its request by a binary
// search in the chunk's prefix sums), so one long request costs no more than
// many short ones. Pass 0 counts the returns (their total fixes where each one
// lands on the free list), pass 1 returns, pass 2 takes.
__global__ void __launch_bounds__(kResizeThreads)
kv_pages_resize_kernel(int batch, int page_size, int max_pages, int n_pages,
                       const int64_t* __restrict__ ctx_len, const int32_t* __restrict__ count,
                       int32_t* block_table, int32_t* held, int32_t* free_pages,
                       int32_t* free_count, int32_t* status) {
  __shared__ long long warp_sums[32];
  __shared__ long long off[kResizeThreads + 1];   // prefix sums of the chunk's moves
  __shared__ int first[kResizeThreads];           // first column that moves
  __shared__ unsigned char bad[kResizeThreads];
  const int tid = threadIdx.x;
  const long long F0 = *free_count;
  const bool list_ok = F0 >= 0 && F0 <= n_pages;

  // (want, held) of request b; a request with a bad length keeps what it has
  auto load = [&](int b, int& want, int& have) -> int {
    want = have = 0;
    if (b >= batch) return 0;
    const long long c = ctx_len[b], n = count ? (long long)count[b] : 0;
    const int h = held[b];
    if (c < 0 || n < 0 || c > (long long)max_pages * page_size - n || h < 0 || h > max_pages)
      return PCT_DEV_BAD_LENGTH;
    want = (int)((c + n + page_size - 1) / page_size);
    have = h;
    return 0;
  };
  // the chunk's request that owns move u
  auto owner = [&](long long u, int n) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (off[mid] <= u) lo = mid; else hi = mid;
    }
    return lo;
  };

  if (!list_ok) {
    for (int b = tid; b < batch; b += blockDim.x) status[b] = PCT_DEV_BAD_COUNT;
    return;
  }
  long long R = 0;   // pages that come back
  for (int c0 = 0; c0 < batch; c0 += kResizeThreads) {
    int want, have;
    const int st = load(c0 + tid, want, have);
    const int ret = have > want ? have - want : 0;
    long long total;
    const long long ex = block_scan(ret, warp_sums, &total);
    const int n = min(kResizeThreads, batch - c0);
    if (total > 0) {   // look the entries over before anything moves
      off[tid] = ex;
      first[tid] = want;
      bad[tid] = 0;
      __syncthreads();
      for (long long u = tid; u < total; u += kResizeThreads) {
        const int r = owner(u, n);
        const int page =
            block_table[(long long)(c0 + r) * max_pages + first[r] + (int)(u - off[r])];
        if (page < 0 || page >= n_pages) bad[r] = 1;
      }
      __syncthreads();
    }
    const int mark = total > 0 && bad[tid] && ret > 0;
    if (c0 + tid < batch) status[c0 + tid] = st | (mark ? PCT_DEV_BAD_PAGE : 0);
    long long good;
    block_scan(mark ? 0 : ret, warp_sums, &good);
    R += good;
  }
  if (F0 + R > n_pages) {   // more pages than there are: nothing moves
    for (int b = tid; b < batch; b += blockDim.x) status[b] = PCT_DEV_BAD_COUNT;
    return;
  }
  if (R > 0) {
    long long base = 0;
    for (int c0 = 0; c0 < batch; c0 += kResizeThreads) {
      int want, have;
      load(c0 + tid, want, have);
      const bool ok = c0 + tid < batch && status[c0 + tid] == 0;
      const int ret = ok && have > want ? have - want : 0;
      long long total;
      const long long ex = block_scan(ret, warp_sums, &total);
      const int n = min(kResizeThreads, batch - c0);
      off[tid] = ex;
      first[tid] = want;
      __syncthreads();
      for (long long u = tid; u < total; u += kResizeThreads) {
        const int r = owner(u, n);
        int32_t* e = block_table + (long long)(c0 + r) * max_pages + first[r] + (int)(u - off[r]);
        free_pages[F0 + R - 1 - (base + u)] = *e;
        *e = -1;
      }
      if (ret > 0) held[c0 + tid] = want;
      base += total;
      __syncthreads();
    }
  }
  const long long F = F0 + R;
  long long base = 0, used = 0;   // needs of earlier requests; pages taken
  for (int c0 = 0; c0 < batch; c0 += kResizeThreads) {
    int want, have;
    load(c0 + tid, want, have);
    const bool ok = c0 + tid < batch && status[c0 + tid] == 0;
    const int need = ok && want > have ? want - have : 0;
    long long total;
    const long long ex = block_scan(need, warp_sums, &total);
    const int n = min(kResizeThreads, batch - c0);
    const bool granted = base + ex + need <= F;
    off[tid] = ex;
    first[tid] = have;
    if (need > 0) {
      if (granted) held[c0 + tid] = want;
      else status[c0 + tid] = PCT_DEV_NO_PAGE;
    }
    // granted requests are a prefix of those in need
    long long got;
    block_scan(granted ? need : 0, warp_sums, &got);
    for (long long u = tid; u < got; u += kResizeThreads) {
      const int r = owner(u, n);
      block_table[(long long)(c0 + r) * max_pages + first[r] + (int)(u - off[r])] =
          free_pages[F - 1 - (base + u)];
    }
    base += total;
    used += got;
    __syncthreads();
  }
  if (tid == 0) *free_count = (int32_t)(F - used);
}

// One thread per token; the first block of a request also looks over the pages
// that the request uses, so every status word has one writer.
__global__ void __launch_bounds__(256)
kv_tree_slots_kernel(int n_stride, int page_size, int max_pages, int n_pages,
                     const int64_t* __restrict__ ctx_len, const int32_t* __restrict__ count,
                     const int32_t* __restrict__ depth, const int32_t* __restrict__ block_table,
                     int64_t* __restrict__ slot, int64_t* __restrict__ pos,
                     int32_t* __restrict__ status) {
  const int b = blockIdx.y, i = blockIdx.x * blockDim.x + threadIdx.x;
  const long long c = ctx_len[b];
  int n = count ? count[b] : n_stride, st = 0;
  if (n < 0 || n > n_stride) st |= PCT_DEV_BAD_COUNT;
  if (c < 0 || (st == 0 && c > (long long)max_pages * page_size - n)) st |= PCT_DEV_BAD_LENGTH;
  if (st) n = 0;
  const int32_t* row = block_table + (long long)b * max_pages;
  if (i < n_stride) {
    long long s = -1, p = -1;
    if (i < n) {
      const unsigned t = (unsigned)(c + i);
      const unsigned col = t / (unsigned)page_size;
      const int page = row[col];
      if (page >= 0 && page < n_pages)
        s = (long long)page * page_size + (t - col * (unsigned)page_size);
      p = c + (depth ? depth[(long long)b * n_stride + i] : i);
    }
    slot[(long long)b * n_stride + i] = s;
    pos[(long long)b * n_stride + i] = p;
  }
  if (blockIdx.x == 0) {
    int bad = 0;
    if (n > 0) {
      const int e = (int)((c + n - 1) / page_size);
      for (int k = (int)(c / page_size) + threadIdx.x; k <= e; k += blockDim.x) {
        const int page = row[k];
        bad |= page < 0 || page >= n_pages;
      }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) status[b] = st | (bad ? PCT_DEV_BAD_PAGE : 0);
  }
}

struct RowGeom {
  int heads, vec;                     // heads, 16-byte pieces per head
  long long page, slot, head;         // cache strides in 16-byte pieces
  int page_size;
};

// A block moves kAppendRows tokens: one thread a token works out where its row comes
// from and goes to, then the block copies 16-byte pieces, a thread one column (K or V,
// head, piece) of several tokens, eight loads before their stores. No division runs
// per piece (with two of 64 bits each, 32 x 1000 tokens of 8 x 128 bf16 took 63 us; this
// takes 44, 5.3 TB/s).
constexpr int kAppendRows = 32;
constexpr int kAppendLoads = 8;
constexpr int kAppendScan = 2048;
__global__ void __launch_bounds__(256)
kv_append_kernel(RowGeom g, int batch, int n_stride, long long n_slots, int cols,
                 const uint4* __restrict__ k_new, const uint4* __restrict__ v_new, long long s_b,
                 long long s_n, long long s_h, const int64_t* __restrict__ slot, uint4* k_cache,
                 uint4* v_cache, int32_t* status) {
  __shared__ long long from[kAppendRows], to[kAppendRows];
  const int tid = threadIdx.x;
  const long long rows = (long long)batch * n_stride, r0 = (long long)blockIdx.x * kAppendRows;
  if (tid < kAppendRows) {
    long long f = 0, t = -1;
    if (r0 + tid < rows) {
      const long long r = r0 + tid, s = slot[r];
      if (s >= 0 && s < n_slots) {
        const long long b = r / n_stride, pg = s / g.page_size;
        f = b * s_b + (r - b * n_stride) * s_n;
        t = pg * g.page + (s - pg * g.page_size) * g.slot;
      }
    }
    from[tid] = f;
    to[tid] = t;
  }
  __syncthreads();
  const int row = g.heads * g.vec, lanes = blockDim.x / cols, r1 = tid / cols;
  if (r1 < lanes) {
    for (int c = tid - r1 * cols; c < 2 * row; c += cols) {
      const bool is_v = c >= row;
      const int q = is_v ? c - row : c, h = q / g.vec, w = q - h * g.vec;
      const uint4* src = (is_v ? v_new : k_new) + h * s_h + w;
      uint4* dst = (is_v ? v_cache : k_cache) + h * g.head + w;
      for (int r = r1; r < kAppendRows; r += kAppendLoads * lanes) {
        uint4 x[kAppendLoads];
#pragma unroll
        for (int j = 0; j < kAppendLoads; ++j)
          if (r + j * lanes < kAppendRows && to[r + j * lanes] >= 0)
            x[j] = ld_stream16(src + from[r + j * lanes]);
#pragma unroll
        for (int j = 0; j < kAppendLoads; ++j)
          if (r + j * lanes < kAppendRows && to[r + j * lanes] >= 0) dst[to[r + j * lanes]] = x[j];
      }
    }
  }
  // status words: short requests by one block each, long ones (already zero) by
  // whichever block holds the bad slot
  if (n_stride <= kAppendScan) {
    for (int b = blockIdx.x; b < batch; b += gridDim.x) {
      int bad = 0;
#pragma unroll 4
      for (int i = tid; i < n_stride; i += 256)
        bad |= slot[(long long)b * n_stride + i] >= n_slots;
      bad = __syncthreads_or(bad);
      if (tid == 0) status[b] = bad ? PCT_DEV_BAD_PAGE : 0;
    }
  } else if (tid < kAppendRows && r0 + tid < rows && slot[r0 + tid] >= n_slots) {
    atomicOr(status + (r0 + tid) / n_stride, PCT_DEV_BAD_PAGE);
  }
}

// A thread owns one 16-byte column of the rows (a layer's K or V, a head, a
// piece) and moves it along the path in order, kMoves loads before their
// stores. In place that is safe: the path rises strictly from at least 1, so
// node path[i] >= i + 1, and a store to place j + 1 (j in this batch or before)
// can only hit a source path[i] = j + 1 with i <= j, which has been read by then.
// Path, table and rows are read one after another, and that latency bounds it: 64
// requests of up to 15 nodes in 16 layers of 8 x 128 bf16, 63 MB, 17 us.
constexpr int kMoves = 8;
constexpr int kPathChunk = 256;
__global__ void __launch_bounds__(128)
kv_commit_kernel(RowGeom g, long long s_layer, int layers, int max_depth, int max_pages,
                 int n_pages, uint4* k_cache, uint4* v_cache,
                 const int32_t* __restrict__ block_table, const int64_t* __restrict__ ctx_len,
                 const int32_t* __restrict__ count, const int32_t* __restrict__ accept_len,
                 const int32_t* __restrict__ accept_path, int64_t* __restrict__ new_len,
                 int32_t* __restrict__ status) {
  __shared__ long long src[kPathChunk], dst[kPathChunk];
  const int b = blockIdx.y, tid = threadIdx.x;
  const long long c = ctx_len[b];
  const int n = count[b], a = accept_len[b];
  const int32_t* path = accept_path + (long long)b * max_depth;
  const int32_t* row = block_table + (long long)b * max_pages;
  int st = 0;
  if (n < 1) st |= PCT_DEV_BAD_COUNT;
  else if (c < 0 || c > (long long)max_pages * g.page_size - n) st |= PCT_DEV_BAD_LENGTH;
  if (a < 0 || a > max_depth) st |= PCT_DEV_BAD_PATH;
  if (st == 0) {
    int bad = 0;
    for (int i = tid; i < a; i += blockDim.x) {
      const int p = path[i], q = i > 0 ? path[i - 1] : 0;
      if (p <= q || p >= n) bad |= PCT_DEV_BAD_PATH;
      else {
        const int ps = row[(unsigned)(c + p) / (unsigned)g.page_size];
        // i + 1 <= path[i] < n when the path rises; beyond the table only if it does not
        const int pd = i + 1 < n ? row[(unsigned)(c + 1 + i) / (unsigned)g.page_size] : -1;
        if (ps < 0 || ps >= n_pages || pd < 0 || pd >= n_pages) bad |= PCT_DEV_BAD_PAGE;
      }
    }
    if (__syncthreads_or(bad & PCT_DEV_BAD_PATH)) st = PCT_DEV_BAD_PATH;
    else if (__syncthreads_or(bad)) st = PCT_DEV_BAD_PAGE;
  }
  if (blockIdx.x == 0 && tid == 0) {
    status[b] = st;
    new_len[b] = st ? c : c + 1 + a;
  }
  if (st) return;
  const int row_pieces = g.heads * g.vec;
  const long long cols = (long long)layers * 2 * row_pieces;
  for (int i0 = 0; i0 < a; i0 += kPathChunk) {
    const int m = min(kPathChunk, a - i0);
    __syncthreads();
    for (int i = tid; i < m; i += blockDim.x) {
      const unsigned s = (unsigned)(c + path[i0 + i]), d = (unsigned)(c + 1 + i0 + i);
      const unsigned ps = s / (unsigned)g.page_size, pd = d / (unsigned)g.page_size;
      src[i] = row[ps] * g.page + (long long)(s - ps * g.page_size) * g.slot;
      dst[i] = row[pd] * g.page + (long long)(d - pd * g.page_size) * g.slot;
    }
    __syncthreads();
    for (long long q = (long long)blockIdx.x * blockDim.x + tid; q < cols;
         q += (long long)gridDim.x * blockDim.x) {
      const int l2 = (int)(q / row_pieces), r = (int)(q - (long long)l2 * row_pieces);
      const int h = r / g.vec, w = r - h * g.vec;
      uint4* base = ((l2 & 1) ? v_cache : k_cache) + (l2 >> 1) * s_layer + h * g.head + w;
      for (int i = 0; i < m; i += kMoves) {
        uint4 x[kMoves];
#pragma unroll
        for (int j = 0; j < kMoves; ++j)
          if (i + j < m) x[j] = base[src[i + j]];
#pragma unroll
        for (int j = 0; j < kMoves; ++j)
          if (i + j < m) base[dst[i + j]] = x[j];
      }
    }
  }
}

RowGeom geom(const kv_cache_desc& d) {
  const int per = d.dtype == PCT_BF16 ? 8 : 4;
  RowGeom g;
  g.heads = d.heads_kv;
  g.vec = d.head_dim / per;
  g.page = d.page_stride / per;
  g.slot = d.slot_stride / per;
  g.head = d.head_stride / per;
  g.page_size = d.page_size;
  return g;
}

}  // namespace

cudaError_t launch_kv_pages_resize(int batch, int page_size, int max_pages, int n_pages,
                                   const int64_t* ctx_len, const int32_t* count,
                                   int32_t* block_table, int32_t* held, int32_t* free_pages,
                                   int32_t* free_count, int32_t* status, cudaStream_t s) {
  TraceScope t(s, "kv_pages_resize");
  kv_pages_resize_kernel<<<1, kResizeThreads, 0, s>>>(batch, page_size, max_pages, n_pages,
                                                      ctx_len, count, block_table, held,
                                                      free_pages, free_count, status);
  return cudaGetLastError();
}

cudaError_t launch_kv_tree_slots(int batch, int n_stride, int page_size, int max_pages,
                                 int n_pages, const int64_t* ctx_len, const int32_t* count,
                                 const int32_t* depth, const int32_t* block_table, int64_t* slot,
                                 int64_t* pos, int32_t* status, cudaStream_t s) {
  TraceScope t(s, "kv_tree_slots");
  const int threads = n_stride >= 256 ? 256 : (n_stride + 31) / 32 * 32;
  kv_tree_slots_kernel<<<dim3((n_stride + threads - 1) / threads, batch), threads, 0, s>>>(
      n_stride, page_size, max_pages, n_pages, ctx_len, count, depth, block_table, slot, pos,
      status);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const kv_cache_desc& d, int batch, int n_stride, const void* k_new,
                             const void* v_new, const int64_t* new_stride, const int64_t* slot,
                             void* k_cache, void* v_cache, int32_t* status, cudaStream_t s) {
  TraceScope t(s, "kv_append");
  const RowGeom g = geom(d);
  const int per = d.dtype == PCT_BF16 ? 8 : 4;
  const int cols = g.heads * g.vec * 2 < 256 ? g.heads * g.vec * 2 : 256;   // columns a pass
  const long long grid = ((long long)batch * n_stride + kAppendRows - 1) / kAppendRows;
  if (n_stride > kAppendScan) {
    const cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int32_t) * batch, s);
    if (e != cudaSuccess) return e;
  }
  kv_append_kernel<<<(unsigned)grid, 256, 0, s>>>(
      g, batch, n_stride, (long long)d.n_pages * d.page_size, cols,
      static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), new_stride[0] / per,
      new_stride[1] / per, new_stride[2] / per, slot, static_cast<uint4*>(k_cache),
      static_cast<uint4*>(v_cache), status);
  return cudaGetLastError();
}

cudaError_t launch_kv_commit(const kv_cache_desc& d, int batch, int layers, int64_t layer_stride,
                             int max_depth, void* k_cache, void* v_cache,
                             const int32_t* block_table, const int64_t* ctx_len,
                             const int32_t* count, const int32_t* accept_len,
                             const int32_t* accept_path, int64_t* new_len, int32_t* status,
                             cudaStream_t s) {
  TraceScope t(s, "kv_commit");
  const RowGeom g = geom(d);
  const int per = d.dtype == PCT_BF16 ? 8 : 4;
  const long long cols = (long long)layers * 2 * g.heads * g.vec;
  const long long want = (cols + 127) / 128;
  const int gx = (int)(want > 1024 ? 1024 : want);
  kv_commit_kernel<<<dim3(gx, batch), 128, 0, s>>>(
      g, layer_stride / per, layers, max_depth, d.max_pages, d.n_pages,
      static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), block_table, ctx_len, count,
      accept_len, accept_path, new_len, status);
  return cudaGetLastError();
}

}  // namespace pct
