// pages.cu -- the pages of a paged cache: reserving, forking, freeing and
// compacting, with their C ABI (declared in include/dcoco.h).
//
// What a pool holds is in the caller's arrays: a table of pages a row, how many
// of its entries a row holds, its tokens, and a count of holders a page.  A
// plan kernel of one block finds pages (lowest first) and writes the moves; a
// second kernel over the whole GPU changes tables and counts and copies the
// moved pages of every plane (K, V, scales; all layers).
//
// The plan is a scan over the counts, 16 KB a step of 1024 threads; a fork stops
// as soon as it has enough free pages.  The copy is bound by HBM: a warp moves
// 4 KB a step, all its loads in flight before the first store.  2000 of 8001 pages of 263
// KB (K, V, scales of 8 layers) compacted: 134 us, 7.8 TB/s with what stays in L2; 48
// of 64 rows freed and forked anew, 33 KB a copied page and layer: 24 us, of which the
// calls' host part and three dependent launches are 17.  48 rows reserve a page each among 8200: 6 us; among
// 2^20, all held but the last: 220 us, the scan.
#include <cuda_runtime.h>

#include <new>

#include "../../include/dcoco.h"
#include "common.cuh"
#include "launch.h"

namespace dc {
namespace {

constexpr int kPlan = 1024;      // threads of the plan
constexpr int kCopy = 256;       // threads of a copying block
constexpr int kUnitVecs = 256;   // vectors of a warp's step: 8 a lane
constexpr int kNoRow = 0x7F7F7F7F;

struct Fork {
  int src, dst, full, tokens;
};
struct Move {
  int src, dst, refs;
};

// Device workspace of a handle (sizes: pages, rows).
struct Work {
  int *err;
  int *moves_n, *forks_n;  // of the call
  int *claim;              // [rows] least call index that names the row (kNoRow between calls)
  int *rank;               // [rows]
  Fork *fork;              // [rows]
  int *need;               // [rows] pages that a row is to get
  int *free_page;          // [pages]
  Move *move;              // [max(pages, rows)]
  int *map;                // [pages] where a page goes, -1: nobody holds it
};

struct Pool {
  int32_t *table, *held, *len, *refs;
  int64_t stride;
  int num_pages, page_size, max_pages, max_rows;
};

struct Plane {
  uint8_t *base;
  int64_t layer_stride, page_stride;  // bytes
  int vecs;                           // vectors of a page in one layer
  int layers, wide;                   // 16-byte vectors, else 4
  int units;                          // steps of a page, all layers
};
struct Planes {
  Plane p[DCOCO_MAX_PLANES];
  int n, units;  // steps of a page over all planes
};

// Exclusive scan of one value a thread; *total receives the sum.
__device__ int block_scan(int v, int *total) {
  __shared__ int s[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(DC_FULL_MASK, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the last call's readers are done
  if (lane == 31) s[warp] = x;
  __syncthreads();
  int w = lane < kPlan / 32 ? s[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(DC_FULL_MASK, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(DC_FULL_MASK, w, 31);
  const int before = __shfl_sync(DC_FULL_MASK, w, warp == 0 ? 0 : warp - 1);
  return x - v + (warp == 0 ? 0 : before);
}

// The `want` lowest pages without a holder, into list.  -> how many there are (at most want)
__device__ int find_free(const int32_t *refs, int pages, int want, int *list) {
  int found = 0;
  for (int p0 = 0; p0 < pages && found < want; p0 += kPlan * 4) {
    const int p = p0 + threadIdx.x * 4;
    int r[4], mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      r[k] = p + k < pages ? refs[p + k] : 1;
      mine += r[k] == 0;
    }
    int all, at = found + block_scan(mine, &all);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (r[k] == 0) {
        if (at < want) list[at] = p + k;
        ++at;
      }
    found += all;
  }
  __syncthreads();
  return min(found, want);
}

__device__ __forceinline__ int pages_of(int tokens, int page_size) { return tokens / page_size + (tokens % page_size > 0); }

// Rows named twice go to the first that names them.
__device__ void claim_rows(const Work &w, const int32_t *rows, int count, int max_rows) {
  for (int i = threadIdx.x; i < count; i += kPlan)
    if (rows[i] >= 0 && rows[i] < max_rows) atomicMin(&w.claim[rows[i]], i);
  __syncthreads();
}
__device__ void unclaim_rows(const Work &w, const int32_t *rows, int count, int max_rows) {
  __syncthreads();
  for (int i = threadIdx.x; i < count; i += kPlan)
    if (rows[i] >= 0 && rows[i] < max_rows) w.claim[rows[i]] = kNoRow;
}

__global__ void __launch_bounds__(kPlan) k_pages_reserve(const Pool q, const Work w, int count, const int32_t *rows,
                                                         const int32_t *want, int32_t *done) {
  int bad = 0, total = 0;
  claim_rows(w, rows, count, q.max_rows);
  for (int i0 = 0; i0 < count; i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    int need = 0;
    bool ok = false;
    if (i < count) {
      const int row = rows[i];
      ok = row >= 0 && row < q.max_rows && w.claim[row] == i && want[i] >= 0;
      if (ok) {
        const int held = q.held[row], pages = pages_of(want[i], q.page_size);
        ok = held >= 0 && held <= q.max_pages && pages <= q.max_pages;
        if (ok) need = min(max(0, pages - held), q.num_pages + 1);
      }
      if (!ok) bad |= kErrBadRow;
    }
    int all;
    const int at = total + block_scan(need, &all);
    if (i < count) w.rank[i] = ok ? at : -1, w.need[i] = need;
    total = min(total + all, q.num_pages + 1);  // (1024 x 2^20 fit)
  }
  __syncthreads();
  const int have = find_free(q.refs, q.num_pages, min(total, q.num_pages), w.free_page);
  // a warp a row
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < count; i += kPlan / 32) {
    const int at = w.rank[i], need = w.need[i];
    const bool ok = at >= 0 && need <= have - min(at, have);
    if (ok && need > 0) {
      const int row = rows[i], held = q.held[row];
      for (int j = lane; j < need; j += 32) {
        const int page = w.free_page[at + j];
        q.table[row * q.stride + held + j] = page;
        q.refs[page] = 1;
      }
      __syncwarp();
      if (lane == 0) q.held[row] = held + need;
    }
    if (at >= 0 && !ok) bad |= kErrNoPages;
    if (done && lane == 0) done[i] = ok;
  }
  unclaim_rows(w, rows, count, q.max_rows);
  if (bad) atomicOr(w.err, bad);
}

__global__ void __launch_bounds__(kPlan) k_pages_fork_plan(const Pool q, const Work w, int count, const int32_t *src,
                                                           const int32_t *dst, int32_t *done) {
  pdl_trigger();
  int bad = 0, total = 0;
  claim_rows(w, dst, count, q.max_rows);
  for (int i0 = 0; i0 < count; i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    int need = 0;
    bool ok = false;
    if (i < count) {
      const int a = src[i], b = dst[i];
      // the row forked into is empty and named once, and the source is not forked into
      ok = a >= 0 && a < q.max_rows && b >= 0 && b < q.max_rows && w.claim[b] == i && w.claim[a] == kNoRow && q.held[b] == 0;
      if (ok) {
        const int n = q.len[a], held = q.held[a];
        ok = n >= 0 && held >= 0 && held <= q.max_pages && pages_of(n, q.page_size) <= held;
        if (ok) {
          need = n % q.page_size > 0;
          w.fork[i] = Fork{a, b, n / q.page_size, n};
        }
      }
      if (!ok) bad |= kErrBadRow;
    }
    int all;
    const int at = total + block_scan(need, &all);
    if (i < count) w.rank[i] = !ok ? -2 : need ? at : -1;  // -2: refused, -1: shares all its pages
    total += all;
  }
  __syncthreads();
  const int have = find_free(q.refs, q.num_pages, min(total, q.num_pages), w.free_page);
  for (int i = threadIdx.x; i < count; i += kPlan) {
    const int at = w.rank[i];
    bool ok = at >= -1 && at < have;
    int fresh = -1;
    if (ok) {
      const Fork f = w.fork[i];
      if (at >= 0) {
        const int from = q.table[f.src * q.stride + f.full];
        fresh = w.free_page[at];
        if (from < 0 || from >= q.num_pages) bad |= kErrBadPage, w.move[at] = Move{-1, -1, 0};
        else w.move[at] = Move{from, fresh, 1};
        q.refs[fresh] = 1;
        q.table[f.dst * q.stride + f.full] = fresh;
      }
      q.held[f.dst] = pages_of(f.tokens, q.page_size);
      q.len[f.dst] = f.tokens;
    } else if (at >= 0) {
      bad |= kErrNoPages;
    }
    if (!ok) w.fork[i].full = w.fork[i].tokens = 0;  // nothing to share
    if (done) done[i] = ok;
  }
  if (threadIdx.x == 0) *w.moves_n = have, *w.forks_n = count;
  unclaim_rows(w, dst, count, q.max_rows);
  if (bad) atomicOr(w.err, bad);
}

// A block a listed row; a row listed twice is freed once.
__global__ void __launch_bounds__(128) k_pages_free(const Pool q, const Work w, const int32_t *rows) {
  __shared__ int s_held;
  const int row = rows[blockIdx.x];
  int bad = 0;
  if (row < 0 || row >= q.max_rows) {
    if (threadIdx.x == 0) atomicOr(w.err, kErrBadRow);
    return;
  }
  if (threadIdx.x == 0) s_held = atomicExch(&q.held[row], 0);
  __syncthreads();
  int held = s_held;
  if (held < 0 || held > q.max_pages) bad |= kErrBadRow, held = held < 0 ? 0 : q.max_pages;
  for (int j = threadIdx.x; j < held; j += 128) {
    const int page = q.table[row * q.stride + j];
    if (page < 0 || page >= q.num_pages) {
      bad |= kErrBadPage;
    } else if (atomicSub(&q.refs[page], 1) <= 0) {
      atomicAdd(&q.refs[page], 1);  // nobody held it
      bad |= kErrBadPage;
    }
  }
  if (threadIdx.x == 0) q.len[row] = 0;
  if (bad) atomicOr(w.err, bad);
}

// Pages in use from `live` on go, in order, to the free ones below it.
__global__ void __launch_bounds__(kPlan) k_pages_compact_plan(const int32_t *refs, int pages, const Work w, int32_t *live_out) {
  pdl_trigger();
  int live = 0;
  for (int p0 = 0; p0 < pages; p0 += kPlan * 4) {
    int mine = 0, all;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p = p0 + k * kPlan + threadIdx.x;
      mine += p < pages && refs[p] > 0;
    }
    block_scan(mine, &all);
    live += all;
  }
  int holes = 0, movers = 0;
  for (int p0 = 0; p0 < pages; p0 += kPlan * 4) {
    const int p = p0 + threadIdx.x * 4;
    bool hole[4], mover[4];
    int mh = 0, mm = 0, all;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = p + k < pages, used = in && refs[p + k] > 0;
      hole[k] = in && !used && p + k < live;
      mover[k] = used && p + k >= live;
      if (in && !mover[k]) w.map[p + k] = used ? p + k : -1;
      mh += hole[k], mm += mover[k];
    }
    int at = holes + block_scan(mh, &all);
    holes += all;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (hole[k]) w.move[at++].dst = p + k;
    at = movers + block_scan(mm, &all);
    movers += all;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (mover[k]) w.move[at].src = p + k, w.move[at++].refs = refs[p + k];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < movers; i += kPlan) w.map[w.move[i].src] = w.move[i].dst;
  if (threadIdx.x == 0) *w.moves_n = movers, *live_out = live;
}

template <typename T>
__device__ __forceinline__ void copy_unit(const Plane &pl, const Move &m, int v0) {
  const int lane = threadIdx.x & 31;
  const uint8_t *src = pl.base + m.src * pl.page_stride;
  uint8_t *dst = pl.base + m.dst * pl.page_stride;
  T x[kUnitVecs / 32];
  int64_t at[kUnitVecs / 32];
  const int all = pl.vecs * pl.layers;
#pragma unroll
  for (int k = 0; k < kUnitVecs / 32; ++k) {
    const int v = v0 + k * 32 + lane, layer = v / pl.vecs;
    at[k] = v < all ? layer * pl.layer_stride + (int64_t)(v - layer * pl.vecs) * (int)sizeof(T) : -1;
    if (at[k] >= 0) x[k] = *reinterpret_cast<const T *>(src + at[k]);
  }
#pragma unroll
  for (int k = 0; k < kUnitVecs / 32; ++k)
    if (at[k] >= 0) *reinterpret_cast<T *>(dst + at[k]) = x[k];
}

// The moved pages, a warp a step of 256 vectors.
__device__ void copy_moves(const Planes &pl, const Work &w) {
  const int64_t total = (int64_t)*w.moves_n * pl.units, warps = (int64_t)gridDim.x * (kCopy / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kCopy / 32) + (threadIdx.x >> 5); u < total; u += warps) {
    const Move m = w.move[u / pl.units];
    int r = (int)(u % pl.units), i = 0;
    while (r >= pl.p[i].units) r -= pl.p[i++].units;
    if (m.src < 0) continue;
    if (pl.p[i].wide) copy_unit<uint4>(pl.p[i], m, r * kUnitVecs);
    else copy_unit<uint32_t>(pl.p[i], m, r * kUnitVecs);
  }
}

__global__ void __launch_bounds__(kCopy) k_pages_fork(const Pool q, const Work w, const __grid_constant__ Planes pl) {
  pdl_wait();
  int bad = 0;
  // the shared pages, a warp a fork
  const int lane = threadIdx.x & 31, forks = *w.forks_n;
  for (int i = blockIdx.x * (kCopy / 32) + (threadIdx.x >> 5); i < forks; i += gridDim.x * (kCopy / 32)) {
    const Fork f = w.fork[i];
    const int pages = pages_of(f.tokens, q.page_size);
    // four entries a lane in flight: the count of each is read before it grows (one entry at a
    // time took 6 us more for 48 forks of up to 500)
    for (int j0 = lane; j0 < pages; j0 += 128) {
      int page[4], refs[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) page[k] = j0 + k * 32 < pages ? q.table[f.src * q.stride + j0 + k * 32] : 0;
      // (counts only grow here, so a page that nobody holds has none for all that look)
#pragma unroll
      for (int k = 0; k < 4; ++k) refs[k] = page[k] >= 0 && page[k] < q.num_pages ? __ldcg(&q.refs[page[k]]) : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = j0 + k * 32;
        if (j < pages && refs[k] <= 0) bad |= kErrBadPage;
        if (j >= f.full) continue;  // (filled in part: copied)
        q.table[f.dst * q.stride + j] = page[k];
        if (refs[k] > 0) atomicAdd(&q.refs[page[k]], 1);
      }
    }
  }
  copy_moves(pl, w);
  if (bad) atomicOr(w.err, bad);
}

__global__ void __launch_bounds__(kCopy) k_pages_compact(const Pool q, const Work w, const __grid_constant__ Planes pl,
                                                         int32_t *table_out, int64_t out_stride, int32_t *refs_out,
                                                         const int32_t *live_p) {
  pdl_wait();
  int bad = 0;
  const int live = *live_p, moves = *w.moves_n, lane = threadIdx.x & 31;
  const int warp = blockIdx.x * (kCopy / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kCopy / 32);
  for (int row = warp; row < q.max_rows; row += warps) {
    int held = q.held[row];
    if (held < 0 || held > q.max_pages) bad |= kErrBadRow, held = held < 0 ? 0 : q.max_pages;
    for (int j = lane; j < held; j += 32) {
      const int page = q.table[row * q.stride + j];
      int to = page;
      if (page >= 0 && page < q.num_pages) to = w.map[page];
      else bad |= kErrBadPage;
      // nobody holds it: left as it is (another page may move there, so it is as wrong as before)
      if (to < 0) bad |= kErrBadPage, to = page;
      table_out[row * out_stride + j] = to;
    }
  }
  const int tid = blockIdx.x * kCopy + threadIdx.x, threads = gridDim.x * kCopy;
  for (int p = tid; p < q.num_pages; p += threads) {
    if (p >= live) refs_out[p] = 0;
    else if (refs_out != q.refs && q.refs[p] > 0) refs_out[p] = q.refs[p];
  }
  for (int i = tid; i < moves; i += threads) refs_out[w.move[i].dst] = w.move[i].refs;
  copy_moves(pl, w);
  if (bad) atomicOr(w.err, bad);
}

}  // namespace
}  // namespace dc

using namespace dc;

struct dcoco_pages_handle {
  dcoco_pages_config cfg;
  int sms = 1;
  void *block = nullptr;
  Work w;
  cudaStream_t last_stream = nullptr;
  long long launches = 0;
};

namespace {

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? DCOCO_OK : DCOCO_ECUDA; }

int check_pool(const dcoco_pages_handle *h, const dcoco_pages_state *s, bool len) {
  if (!h || !s) return DCOCO_EINVAL;
  if (!s->page_table || !s->held || !s->refs || (len && !s->len)) return DCOCO_EINVAL;
  if (s->page_table_stride < h->cfg.max_pages) return DCOCO_EINVAL;
  return DCOCO_OK;
}

Pool make_pool(const dcoco_pages_handle *h, const dcoco_pages_state *s) {
  const dcoco_pages_config &c = h->cfg;
  return Pool{s->page_table, s->held, s->len, s->refs, s->page_table_stride, c.num_pages, c.page_size, c.max_pages, c.max_rows};
}

// Planes whose pages lie apart from one another, in whole vectors.
int make_planes(const dcoco_pages_handle *h, int n, const dcoco_page_plane *planes, Planes *out) {
  if (n < 0 || n > DCOCO_MAX_PLANES || (n > 0 && !planes)) return DCOCO_EINVAL;
  out->n = n, out->units = 0;
  const int64_t pages = h->cfg.num_pages;
  int64_t units = 0;
  for (int i = 0; i < n; ++i) {
    const dcoco_page_plane &a = planes[i];
    const int64_t ls = a.layer_stride, ps = a.page_stride, b = a.page_bytes;
    if (!a.base || a.layers < 1 || a.layers > 65536 || b < 4 || b > (1ll << 30)) return DCOCO_EINVAL;
    if ((a.layers > 1 && (ls < b || ls > (1ll << 46))) || (pages > 1 && (ps < b || ps > (1ll << 46)))) return DCOCO_EINVAL;
    if (a.layers > 1 && pages > 1 && ls < (pages - 1) * ps + b && ps < (a.layers - 1) * ls + b) return DCOCO_EINVAL;
    const int64_t all = (int64_t)(reinterpret_cast<uintptr_t>(a.base)) | b | (a.layers > 1 ? ls : 0) | (pages > 1 ? ps : 0);
    if (all % 4 != 0) return DCOCO_EINVAL;
    const int wide = all % 16 == 0;
    const int64_t vecs = b / (wide ? 16 : 4);
    if (vecs * a.layers > (1ll << 30)) return DCOCO_EINVAL;
    const int u = (int)((vecs * a.layers + kUnitVecs - 1) / kUnitVecs);
    out->p[i] = Plane{static_cast<uint8_t *>(a.base), a.layers > 1 ? ls : 0, pages > 1 ? ps : 0, (int)vecs, a.layers, wide, u};
    units += u;
  }
  if (units > (1ll << 30)) return DCOCO_EINVAL;
  out->units = (int)units;
  return DCOCO_OK;
}

// Blocks that a copy of up to `moves` pages fills, at most eight an SM.
unsigned copy_grid(const dcoco_pages_handle *h, const Planes &pl, int64_t moves, int64_t other_warps) {
  const int64_t warps = moves * pl.units > other_warps ? moves * pl.units : other_warps;
  const int64_t blocks = (warps + kCopy / 32 - 1) / (kCopy / 32), most = 8ll * h->sms;
  return (unsigned)(blocks < 1 ? 1 : blocks < most ? blocks : most);
}

}  // namespace

extern "C" {

int dcoco_pages_create(const dcoco_pages_config *cfg, dcoco_pages_handle **out) {
  if (!cfg || !out) return DCOCO_EINVAL;
  const dcoco_pages_config &c = *cfg;
  if (c.num_pages < 1 || c.num_pages > (1 << 20) || c.max_pages < 1 || c.max_rows < 1 || c.max_rows > (1 << 20) ||
      c.page_size < 1 || (int64_t)c.page_size * c.max_pages > (1ll << 30))
    return DCOCO_EINVAL;
  dcoco_pages_handle *h = new (std::nothrow) dcoco_pages_handle();
  if (!h) return DCOCO_ENOMEM;
  h->cfg = c;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
    delete h;
    return DCOCO_ECUDA;
  }
  const size_t pages = c.num_pages, rows = c.max_rows, moves = pages > rows ? pages : rows;
  const auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t claim = 256, rank = claim + up(rows * 4), fork = rank + up(rows * 4), need = fork + up(rows * sizeof(Fork)),
               freep = need + up(rows * 4), move = freep + up(pages * 4), map = move + up(moves * sizeof(Move)),
               bytes = map + up(pages * 4);
  if (cudaMalloc(&h->block, bytes) != cudaSuccess) {
    cudaGetLastError();
    delete h;
    return DCOCO_ENOMEM;
  }
  char *b = static_cast<char *>(h->block);
  h->w = Work{(int *)b, (int *)(b + 8), (int *)(b + 12), (int *)(b + claim), (int *)(b + rank), (Fork *)(b + fork),
              (int *)(b + need), (int *)(b + freep), (Move *)(b + move), (int *)(b + map)};
  if (cudaMemset(b, 0, 256) != cudaSuccess || cudaMemset(b + claim, 0x7F, rows * 4) != cudaSuccess ||
      cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    cudaFree(h->block);
    delete h;
    return DCOCO_ECUDA;
  }
  *out = h;
  return DCOCO_OK;
}

int dcoco_pages_reserve(dcoco_pages_handle *h, const dcoco_pages_state *s, int count, const int32_t *rows,
                        const int32_t *tokens, int32_t *done, void *stream) {
  const int rc = check_pool(h, s, false);
  if (rc != DCOCO_OK) return rc;
  if (count < 0 || count > h->cfg.max_rows) return DCOCO_EBATCH;
  if (count == 0) return DCOCO_OK;
  if (!rows || !tokens) return DCOCO_EINVAL;
  h->last_stream = static_cast<cudaStream_t>(stream);
  ++h->launches;
  k_pages_reserve<<<1, kPlan, 0, h->last_stream>>>(make_pool(h, s), h->w, count, rows, tokens, done);
  return cuda_status(cudaGetLastError());
}

int dcoco_pages_fork(dcoco_pages_handle *h, const dcoco_pages_state *s, int planes_n, const dcoco_page_plane *planes,
                     int count, const int32_t *src, const int32_t *dst, int32_t *done, void *stream) {
  int rc = check_pool(h, s, true);
  if (rc != DCOCO_OK) return rc;
  if (count < 0 || count > h->cfg.max_rows) return DCOCO_EBATCH;
  Planes pl;
  rc = make_planes(h, planes_n, planes, &pl);
  if (rc != DCOCO_OK) return rc;
  if (count == 0) return DCOCO_OK;
  if (!src || !dst) return DCOCO_EINVAL;
  h->last_stream = static_cast<cudaStream_t>(stream);
  h->launches += 2;
  const Pool q = make_pool(h, s);
  k_pages_fork_plan<<<1, kPlan, 0, h->last_stream>>>(q, h->w, count, src, dst, done);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_ex(k_pages_fork, dim3(copy_grid(h, pl, count, count)), dim3(kCopy), 0, h->last_stream, true, 0,
                               q, h->w, pl));
}

int dcoco_pages_free(dcoco_pages_handle *h, const dcoco_pages_state *s, int count, const int32_t *rows, void *stream) {
  const int rc = check_pool(h, s, true);
  if (rc != DCOCO_OK) return rc;
  if (count < 0 || count > h->cfg.max_rows) return DCOCO_EBATCH;
  if (count == 0) return DCOCO_OK;
  if (!rows) return DCOCO_EINVAL;
  h->last_stream = static_cast<cudaStream_t>(stream);
  ++h->launches;
  k_pages_free<<<count, 128, 0, h->last_stream>>>(make_pool(h, s), h->w, rows);
  return cuda_status(cudaGetLastError());
}

int dcoco_pages_compact(dcoco_pages_handle *h, const dcoco_pages_state *s, int planes_n, const dcoco_page_plane *planes,
                        int32_t *table_out, int64_t table_out_stride, int32_t *refs_out, int32_t *live, void *stream) {
  int rc = check_pool(h, s, false);
  if (rc != DCOCO_OK) return rc;
  if (!table_out || !refs_out || !live || table_out_stride < h->cfg.max_pages) return DCOCO_EINVAL;
  if (table_out == s->page_table && table_out_stride != s->page_table_stride) return DCOCO_EINVAL;
  Planes pl;
  rc = make_planes(h, planes_n, planes, &pl);
  if (rc != DCOCO_OK) return rc;
  h->last_stream = static_cast<cudaStream_t>(stream);
  h->launches += 2;
  k_pages_compact_plan<<<1, kPlan, 0, h->last_stream>>>(s->refs, h->cfg.num_pages, h->w, live);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e);
  const int64_t other = h->cfg.max_rows > h->cfg.num_pages / 32 ? h->cfg.max_rows : h->cfg.num_pages / 32;
  return cuda_status(launch_ex(k_pages_compact, dim3(copy_grid(h, pl, (h->cfg.num_pages + 1) / 2, other)), dim3(kCopy), 0,
                               h->last_stream, true, 0, make_pool(h, s), h->w, pl, table_out, table_out_stride, refs_out,
                               (const int32_t *)live));
}

int dcoco_pages_status(dcoco_pages_handle *h) {
  if (!h) return DCOCO_EINVAL;
  if (cudaStreamSynchronize(h->last_stream) != cudaSuccess) return DCOCO_ECUDA;
  int flag = 0;
  if (cudaMemcpy(&flag, h->w.err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return DCOCO_ECUDA;
  if (flag != 0) {
    if (cudaMemset(h->w.err, 0, sizeof(int)) != cudaSuccess) return DCOCO_ECUDA;
    return DCOCO_EDEVICE;
  }
  return DCOCO_OK;
}

long long dcoco_pages_launches(const dcoco_pages_handle *h) { return h ? h->launches : -1; }

void dcoco_pages_destroy(dcoco_pages_handle *h) {
  if (!h) return;
  cudaDeviceSynchronize();
  cudaFree(h->block);
  delete h;
}

}  // extern "C"
