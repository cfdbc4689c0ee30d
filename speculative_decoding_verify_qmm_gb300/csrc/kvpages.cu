// Pages of the paged KV cache: shared between requests (fork), made exclusive where a round will write, grown, trimmed and
// freed (reserve), moved to the front (compact), handed to another cache (copy).
//
// The only state is a count of the table entries that name each page; a page without any is free, and the lowest free pages
// are taken first: every result follows from the inputs, whatever the order in which threads run.
//
// Bookkeeping is bound by latency (a chain of lookups: request, table entry, count), the copies by memory.  So each call is
// one CTA that decides everything - a scan of the counts with 64 bytes a thread, no traffic between SMs - and one launch of
// all SMs that moves the bytes and does what needs no order (counts going down, tables renumbered).
//
// Measured (8 key heads of 128, us in a graph): 8 samples of a prompt of 5000 tokens forked, reserved for 8 rows (8-bit, 36 layers) and
// freed 21; 96 samples of three prompts of 1511 tokens, bf16, 64 layers 74; 945 of 3000 pages moved in 36 layers, 4-bit, 161 (5.5 TB/s); 257 pages of
// 64 tokens handed over in 36 layers, 8-bit, 394 to 414 (6.4 TB/s of the 6.8 that a copy reaches).
#include "sv_kv.cuh"

#include <algorithm>
#include <cstring>
#include <functional>

namespace sv {

constexpr int PG_THREADS = 1024, PG_WARPS = PG_THREADS / 32;
constexpr int PG_SCAN = 16;                         // counts a thread looks at in one step of a scan
constexpr int PG_LAYERS = 64;                       // caches per launch: their pointers ride in the launch parameters
constexpr int PC_THREADS = 256;                     // of a copying CTA
constexpr int PC_STAGES = 6, PC_LEAD = 4;           // whole pages: tiles of a warp in shared memory, and on their way in
constexpr int PC_SMEM = 192 * 1024;                 // of all its warps that copy

struct PagePool {
  int32_t *refs, *table, *held;
  int n_pages, page_shift, slots, table_pages;
};

struct ReserveParams {
  PagePool g;
  const int32_t *keep, *need;
  int32_t *counts, *copies;
  int32_t* list;        // [n_pages] workspace: pages handed out, then what they replace (plus 1)
  int32_t* before;      // [slots] workspace: pages that a slot held, where it gives some back
};

struct PageCopyParams {
  KvPtrs from[PG_LAYERS], to[PG_LAYERS];
  KvCache c;                             // sizes (pointers unused)
  int n_layers, to_pages;
  const int32_t *src, *dst, *places;     // of copy i: at i * step; places NULL = whole pages
  int step, n;                           // copies, or at most so many
  const int32_t* count;                  // DEVICE: copies (NULL: n)
  int tiles_kv, tiles;                   // tiles of K (and of V), and of all arrays of a page
  int stage;                             // whole pages: bytes of a tile
  int side_tiles;                        // tiles of each array of scales or biases; 0: the four share one
  // after a reserve or a compact: what is left of the bookkeeping
  PagePool g;
  int32_t *list, *before;
  const int32_t *fresh;                  // entries of list
  const int32_t* live;                   // pages in use after a compact
};

// Exclusive prefix of `v` over the CTA's threads and the total, by all threads.
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int s_warp[PG_WARPS + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += up;
  }
  __syncthreads();                       // the last call's results have been read
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int mine = s_warp[lane];
    int t = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, t, off);
      if (lane >= off) t += up;
    }
    s_warp[lane] = t - mine;
    if (lane == 31) s_warp[PG_WARPS] = t;
  }
  __syncthreads();
  *total = s_warp[PG_WARPS];
  return s_warp[warp] + inc - v;
}

// Bit i: count first + i is zero (free pages) or not, for the pages of [lo, hi).
__device__ __forceinline__ unsigned page_bits(const int32_t* refs, int first, int lo, int hi, bool free) {
  unsigned m = 0;
  if (first + PG_SCAN <= hi && first >= lo && (reinterpret_cast<uintptr_t>(refs + first) & 15) == 0) {
    int4 x[PG_SCAN / 4];
#pragma unroll
    for (int i = 0; i < PG_SCAN / 4; ++i) x[i] = reinterpret_cast<const int4*>(refs + first)[i];
#pragma unroll
    for (int i = 0; i < PG_SCAN / 4; ++i)
      m |= (unsigned)(x[i].x == 0) << (4 * i) | (unsigned)(x[i].y == 0) << (4 * i + 1) | (unsigned)(x[i].z == 0) << (4 * i + 2) |
           (unsigned)(x[i].w == 0) << (4 * i + 3);
    return free ? m : ~m & ((1u << PG_SCAN) - 1);
  }
  for (int i = 0; i < PG_SCAN; ++i) {
    const int p = first + i;
    if (p >= lo && p < hi && (refs[p] == 0) == free) m |= 1u << i;
  }
  return m;
}

// The pages of [lo, hi) that are free (or are not), in order, to put(rank, page), until `most` are found; how many there are (up
// to the end of the step that had the last).
template <typename Put>
__device__ __forceinline__ int page_scan(const int32_t* refs, int lo, int hi, bool free, int most, Put put) {
  int found = 0;
  for (int base = lo & ~3; base < hi && found < most; base += PG_THREADS * PG_SCAN) {
    const int first = base + threadIdx.x * PG_SCAN;
    unsigned m = first < hi ? page_bits(refs, first, lo, hi, free) : 0u;
    int total;
    int rank = found + block_scan(__popc(m), &total);
    for (; m; m &= m - 1, ++rank)
      if (rank < most) put(rank, first + __ffs(m) - 1);
    found += total;
  }
  return found;
}

// ------------------------------------------------------------------- fork
__global__ void __launch_bounds__(128) kv_fork_kernel(PagePool g, int n, const int32_t* parents, const int32_t* children, const int32_t* tokens) {
  pdl_trigger();
  pdl_wait();
  const int f = blockIdx.x, p = parents[f], c = children[f], t = tokens[f];
  bool bad = (unsigned)p >= (unsigned)g.slots || (unsigned)c >= (unsigned)g.slots || p == c || t < 0;
  // of two forks into one slot the first stands; a slot that is filled here is nobody's parent (its pages would depend on the order)
  for (int i = threadIdx.x; i < n; i += blockDim.x) bad |= (i < f && children[i] == c) || children[i] == p;
  bad = __syncthreads_or(bad);
  int pages = 0;
  if (!bad) {
    const int has = g.held[p];
    pages = (int)(((long long)t + (1 << g.page_shift) - 1) >> g.page_shift);
    bad = g.held[c] != 0 || pages > has || has > g.table_pages;
    if (!bad)
      for (int e = threadIdx.x; e < pages; e += blockDim.x) bad |= (unsigned)g.table[(size_t)p * g.table_pages + e] >= (unsigned)g.n_pages;
    bad = __syncthreads_or(bad);
  }
  if (bad) {
    if (threadIdx.x == 0) raise_error(ERR_BAD_INPUT);
    return;
  }
  for (int e = threadIdx.x; e < pages; e += blockDim.x) {
    const int id = g.table[(size_t)p * g.table_pages + e];
    g.table[(size_t)c * g.table_pages + e] = id;
    atomicAdd(g.refs + id, 1);
  }
  if (threadIdx.x == 0) g.held[c] = pages;
}

// ---------------------------------------------------------------- reserve
// What an entry of a slot needs.
struct PageEntry {
  int slot, e, id;       // id: the page there, or -1
  bool shared, part;     // more than one entry names it; it is the half-filled page
};

__global__ void __launch_bounds__(PG_THREADS, 1) kv_reserve_kernel(const __grid_constant__ ReserveParams p) {
  // per slot: first entry that will be written (-1: the slot is left alone), entries before and after, places of the half-filled page
  __shared__ int s_first[MAX_BATCH], s_has[MAX_BATCH], s_wants[MAX_BATCH], s_part[MAX_BATCH], s_bad[MAX_BATCH];
  __shared__ __align__(16) int s_asks[MAX_BATCH];     // the half-filled page if others name it too, or -1
  __shared__ int s_copy[MAX_BATCH];                   // number of its copy, or -1
  __shared__ int s_before[MAX_BATCH + 1];             // entries to look at before the slot's
  pdl_trigger();
  pdl_wait();
  const PagePool& g = p.g;
  const int tid = threadIdx.x, page = 1 << g.page_shift;
  int look = 0;
  if (tid < MAX_BATCH) {
    int first = -1, has = 0, wants = 0, part = 0;
    if (tid < g.slots) {
      const int keep = p.keep[tid], need = p.need[tid];
      has = g.held[tid];
      if (need >= 0) {
        wants = (int)(((long long)need + page - 1) >> g.page_shift);
        if (has < 0 || has > g.table_pages || keep < 0 || keep > need || (long long)keep > (long long)has << g.page_shift || wants > g.table_pages) {
          raise_error(ERR_BAD_INPUT);
        } else {
          first = keep >> g.page_shift;
          part = keep & (page - 1);
          look = max(0, wants - first);
        }
      }
    }
    s_first[tid] = first;
    s_has[tid] = has;
    s_wants[tid] = wants;
    s_part[tid] = part;
    s_asks[tid] = s_copy[tid] = -1;
    s_bad[tid] = 0;
    if (tid < g.slots) p.before[tid] = 0;             // the workspace may hold anything; the next launch looks at every slot
  }
  int entries;
  const int mine = block_scan(look, &entries);
  if (tid < MAX_BATCH) s_before[tid] = mine;
  if (tid == 0) s_before[MAX_BATCH] = entries;
  __syncthreads();
  // entry x of all those that will be written, in slot and entry order
  auto entry = [&](int x) {
    int lo = 0, hi = MAX_BATCH;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_before[mid] <= x) lo = mid; else hi = mid;
    }
    PageEntry y;
    y.slot = lo;
    y.e = s_first[lo] + x - s_before[lo];
    y.id = y.e < s_has[lo] ? g.table[(size_t)lo * g.table_pages + y.e] : -1;
    y.part = y.e == s_first[lo] && s_part[lo] > 0;
    y.shared = false;
    if (y.e < s_has[lo]) {
      if ((unsigned)y.id >= (unsigned)g.n_pages) s_bad[lo] = 1;
      else y.shared = g.refs[y.id] > 1;
    }
    return y;
  };
  auto fresh = [&](const PageEntry& y) {
    return !s_bad[y.slot] && (y.e >= s_has[y.slot] || (y.shared && (!y.part || s_copy[y.slot] >= 0)));
  };
  // Entries that go back are judged before anything is changed, too: a warp has a slot's next 128 on their way at once.  (96 samples
  // forked, reserved and freed: 74.0 us, 71.9 without the look; four slots a warp at once no faster.)
#pragma unroll 1
  for (int s = tid >> 5; s < g.slots; s += PG_WARPS) {
    const int has = s_first[s] < 0 ? 0 : s_has[s];
    const int32_t* row = g.table + (size_t)s * g.table_pages;
#pragma unroll 1
    for (int e = s_wants[s] + (tid & 31); e < has; e += 128) {
      int id[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) id[y] = e + 32 * y < has ? row[e + 32 * y] : 0;
      bool bad = false;
#pragma unroll
      for (int y = 0; y < 4; ++y) bad |= (unsigned)id[y] >= (unsigned)g.n_pages;
      if (bad) s_bad[s] = 1;
    }
  }
  // half-filled pages that others name too
  for (int x = tid; x < entries; x += PG_THREADS) {
    const PageEntry y = entry(x);
    if (y.part && y.shared) s_asks[y.slot] = y.id;
  }
  __syncthreads();
  bool copies = false;
  if (tid < MAX_BATCH) {
    if (s_bad[tid]) {
      raise_error(ERR_BAD_INPUT);
      s_asks[tid] = -1;
    }
  }
  __syncthreads();
  if (tid < MAX_BATCH && s_asks[tid] >= 0) {
    // where every entry that names the page asks for it, the first of them keeps it
    const int id = s_asks[tid];
    int same = 0, lower = 0;
    for (int t = 0; t < g.slots; t += 4) {
      const int4 v = *reinterpret_cast<const int4*>(s_asks + t);
      const int n0 = v.x == id, n1 = v.y == id, n2 = v.z == id, n3 = v.w == id;
      same += n0 + n1 + n2 + n3;
      lower += (n0 && t < tid) + (n1 && t + 1 < tid) + (n2 && t + 2 < tid) + (n3 && t + 3 < tid);
    }
    copies = lower > 0 || same != g.refs[id];
  }
  int n_copies;
  const int number = block_scan(copies, &n_copies);
  if (copies) s_copy[tid] = number;
  __syncthreads();
  // how many pages are wanted, and the lowest free ones
  int want = 0;
  for (int x = tid; x < entries; x += PG_THREADS) want += fresh(entry(x));
  int wanted;
  block_scan(want, &wanted);
  int32_t* const list = p.list;
  const int found = min(wanted, page_scan(g.refs, 0, g.n_pages, true, wanted, [&](int rank, int id) { list[rank] = id; }));
  __syncthreads();
  if (found < wanted) {                               // too few: nothing is changed
    for (int i = tid; i < found; i += PG_THREADS) list[i] = 0;
    if (tid == 0) {
      p.counts[0] = wanted - found;
      p.counts[1] = p.counts[2] = 0;
    }
    return;
  }
  // Counts that go down wait for the next launch: every entry is judged by the counts before the call.
  int done = 0;
  for (int x0 = 0; x0 < entries; x0 += PG_THREADS) {
    const int x = x0 + tid;
    PageEntry y;
    bool take = false;
    if (x < entries) {
      y = entry(x);
      take = fresh(y);
    }
    int total;
    const int rank = done + block_scan(take, &total);
    done += total;
    if (take) {
      const int id = list[rank];
      list[rank] = y.e < s_has[y.slot] ? y.id + 1 : 0;
      g.refs[id] = 1;
      g.table[(size_t)y.slot * g.table_pages + y.e] = id;
      if (y.part && y.e < s_has[y.slot]) {
        int32_t* to = p.copies + 3 * s_copy[y.slot];
        to[0] = y.id;
        to[1] = id;
        to[2] = s_part[y.slot];
      }
    }
  }
  if (tid < g.slots && s_first[tid] >= 0 && !s_bad[tid]) {
    g.held[tid] = s_wants[tid];
    if (s_has[tid] > s_wants[tid]) p.before[tid] = s_has[tid];
  }
  if (tid == 0) {
    p.counts[0] = 0;
    p.counts[1] = n_copies;
    p.counts[2] = wanted;
  }
}

// ---------------------------------------------------------------- compact
__global__ void __launch_bounds__(PG_THREADS, 1) kv_compact_kernel(PagePool g, int32_t* counts, int32_t* moves) {
  pdl_trigger();
  pdl_wait();
  const int live = page_scan(g.refs, 0, g.n_pages, false, 0x7fffffff, [](int, int) {});
  const int holes = page_scan(g.refs, 0, live, true, 0x7fffffff, [&](int rank, int id) { moves[2 * rank + 1] = id; });
  page_scan(g.refs, live, g.n_pages, false, 0x7fffffff, [&](int rank, int id) { moves[2 * rank] = id; });
  __syncthreads();
  for (int i = threadIdx.x; i < holes; i += PG_THREADS) {
    const int from = moves[2 * i], to = moves[2 * i + 1];
    g.refs[to] = g.refs[from];
    g.refs[from] = 0;
  }
  if (threadIdx.x == 0) {
    counts[0] = live;
    counts[1] = holes;
  }
}

// ------------------------------------------------------------------- copy
__device__ __forceinline__ void drop_page(const PagePool& g, int id) {
  if ((unsigned)id < (unsigned)g.n_pages) atomicSub(g.refs + id, 1);
  else raise_error(ERR_BAD_INPUT);
}

// The rest of a reserve: counts of pages that were replaced or given back.
__device__ __forceinline__ void finish_reserve(const PageCopyParams& p) {
  const int at = blockIdx.x * PC_THREADS + threadIdx.x, all = gridDim.x * PC_THREADS;
  for (int i = at, n = *p.fresh; i < n; i += all) {
    const int old = p.list[i];
    if (old) {
      p.list[i] = 0;
      drop_page(p.g, old - 1);
    }
  }
  for (int s = blockIdx.x; s < p.g.slots; s += gridDim.x) {
    const int before = p.before[s], now = p.g.held[s];
    __syncthreads();
    if (before == 0) continue;
    if (threadIdx.x == 0) p.before[s] = 0;
    for (int e = now + threadIdx.x; e < before; e += PC_THREADS) drop_page(p.g, p.g.table[(size_t)s * p.g.table_pages + e]);
  }
}

// The rest of a compact: tables.  src and dst of the moves ascend; a page from live on is in use if it is a src, one below if it is no
// dst (then it was free, and holds another's tokens now).
__device__ __forceinline__ void finish_compact(const PageCopyParams& p) {
  const int live = *p.live, n = *p.count;
  for (int s = blockIdx.x; s < p.g.slots; s += gridDim.x) {
    const int has = p.g.held[s];
    if (has < 0 || has > p.g.table_pages) {
      if (threadIdx.x == 0) raise_error(ERR_BAD_INPUT);
      continue;
    }
    for (int e = threadIdx.x; e < has; e += PC_THREADS) {
      int32_t* at = p.g.table + (size_t)s * p.g.table_pages + e;
      const int id = *at;
      const bool stays = (unsigned)id < (unsigned)live;
      const int32_t* col = stays ? p.dst : p.src;
      int lo = 0, hi = n;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (col[2 * mid] <= id) lo = mid; else hi = mid;
      }
      const bool found = n && col[2 * lo] == id;
      if (found == stays) raise_error(ERR_BAD_INPUT);
      else if (found) *at = p.dst[2 * lo];
    }
  }
}

// ---- beginnings of pages (copies of a reserve): pieces of 16 bytes by threads.  Strided pieces of a few KB are
// nothing for bulk copies (93 copies of 7 places in 64 layers: 61 us by threads, 77 by bulk copies of each head's).
constexpr int PP_AHEAD = 8, PP_TILE = PC_THREADS * PP_AHEAD;   // pieces a thread has in flight; of a tile
// CTAs an SM: three are the better for few copies, two for many, so it is the middle one.  (7 copies of 8 places in 36 layers, with the calls
// around them: 2 22.1 us, 3 21.5; 93 copies of 7 places in 64 layers 2 70.9, 3 74.1, 4 90.9.)
constexpr int PP_CTAS = 3;
template <bool REST>
__global__ void __launch_bounds__(PC_THREADS, PP_CTAS) kv_part_copy_kernel(const __grid_constant__ PageCopyParams p) {
  pdl_trigger();
  pdl_wait();
  if constexpr (REST) finish_reserve(p);
  const int n = p.count ? *p.count : p.n, tid = threadIdx.x;
  const int page = 1 << p.c.page_shift, row16 = p.c.dim * p.c.bits / 128, groups = p.c.dim / GROUP;
  const long long all = (long long)n * p.n_layers * p.tiles;
  for (long long t = blockIdx.x; t < all; t += gridDim.x) {
    const long long pl = t / p.tiles;
    const int tile = (int)(t - pl * p.tiles), i = (int)(pl / p.n_layers), layer = (int)(pl - (long long)i * p.n_layers);
    const int src = p.src[(size_t)i * p.step], dst = p.dst[(size_t)i * p.step], places = p.places[(size_t)i * p.step];
    if ((unsigned)src >= (unsigned)p.c.n_pages || (unsigned)dst >= (unsigned)p.to_pages || (unsigned)places > (unsigned)page) {
      if (tid == 0) raise_error(ERR_BAD_INPUT);
      continue;
    }
    const KvPtrs &from = p.from[layer], &to = p.to[layer];
    if (tile < 2 * p.tiles_kv) {
      const bool is_v = tile >= p.tiles_kv;
      const unsigned per = places * row16, pieces = p.c.heads * per, base = (unsigned)(is_v ? tile - p.tiles_kv : tile) * PP_TILE + tid;
      const size_t page16 = (size_t)p.c.heads * page * row16;
      const uint4* a = reinterpret_cast<const uint4*>(is_v ? from.v : from.k) + src * page16;
      uint4* b = reinterpret_cast<uint4*>(is_v ? to.v : to.k) + dst * page16;
      uint4 x[PP_AHEAD];
      unsigned at[PP_AHEAD];
#pragma unroll
      for (int y = 0; y < PP_AHEAD; ++y) {
        const unsigned k = base + y * PC_THREADS;
        if (k >= pieces) continue;
        at[y] = k / per * (page * row16) + k % per;
        x[y] = a[at[y]];
      }
#pragma unroll
      for (int y = 0; y < PP_AHEAD; ++y)
        if (base + y * PC_THREADS < pieces) b[at[y]] = x[y];
    } else {
      // scales and biases, two bytes at a time: 1/32 or 1/16 of the codes
      const int per = places * groups, pieces = p.c.heads * per;
      const size_t page2 = (size_t)p.c.heads * page * groups, a = src * page2, b = dst * page2;
      for (int k = tid; k < pieces; k += PC_THREADS) {
        const size_t at = (size_t)(k / per) * (page * groups) + k % per;
        const __half s = from.ks[a + at], t2 = from.kb[a + at], u = from.vs[a + at], v = from.vb[a + at];
        to.ks[b + at] = s;
        to.kb[b + at] = t2;
        to.vs[b + at] = u;
        to.vb[b + at] = v;
      }
    }
  }
}

// ---- whole pages: a warp moves tiles of up to PC_STAGE bytes through shared memory with bulk copies, PC_LEAD of them on their way in while
// those before are on their way out.  Tiles of 16 KB and two warps where an array's page has as much (257 pages of 64 KB in 36 layers: 394
// us against 407), of 8 KB and four warps otherwise (pages of 8 KB: 161 against 210).
struct PageTile {
  int layer, src, dst, tile;             // tile < 0: nothing to do
};

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// This lane's piece of a tile: its place in the arrays and in the stage, and its bytes (a multiple of 16, perhaps 0); all: the tile's.
struct PagePiece {
  size_t from, to;                       // byte offsets in the arrays
  uint32_t at, bytes, all;
  int array;                             // K, V, then their scales and biases
};
template <int PC_STAGE>
__device__ __forceinline__ PagePiece page_piece(const PageCopyParams& p, const PageTile& t, int lane) {
  PagePiece x = {};
  if (t.tile < 0) return x;
  const int page = 1 << p.c.page_shift;
  const bool kv = t.tile < 2 * p.tiles_kv;
  const size_t size = (size_t)p.c.heads * page * (kv ? p.c.dim * p.c.bits / 8 : p.c.dim / GROUP * 2);   // of an array's page
  size_t off = 0;
  if (!kv && p.side_tiles == 0) {        // all four arrays at once, a lane each
    x.array = 2 + (lane & 3);
    x.all = (uint32_t)(4 * size);
    x.bytes = lane < 4 ? (uint32_t)size : 0;
    x.at = (uint32_t)((lane & 3) * size);
  } else {
    const int per = kv ? p.tiles_kv : p.side_tiles, tile = kv ? t.tile : t.tile - 2 * p.tiles_kv, a = tile / per;
    x.array = kv ? a : 2 + a;
    off = (size_t)(tile - a * per) * PC_STAGE;
    x.all = size - off < PC_STAGE ? (uint32_t)(size - off) : PC_STAGE;
    x.bytes = lane == 0 ? x.all : 0;
  }
  x.from = t.src * size + off;
  x.to = t.dst * size + off;
  return x;
}
__device__ __forceinline__ uint8_t* page_array(const KvPtrs& c, int array) {
  return array == 0 ? c.k : array == 1 ? c.v : reinterpret_cast<uint8_t*>(array == 2 ? c.ks : array == 3 ? c.kb : array == 4 ? c.vs : c.vb);
}

template <int PC_STAGE, bool REST>
__global__ void __launch_bounds__(PC_THREADS, 1) kv_page_copy_kernel(const __grid_constant__ PageCopyParams p) {
  constexpr int PC_WARPS = PC_SMEM / (PC_STAGES * PC_STAGE);
  static_assert(PC_WARPS <= PC_THREADS / 32 && PC_LEAD < PC_STAGES, "warps, and a stage to store from");
  extern __shared__ __align__(128) uint8_t s_stage[];   // [PC_WARPS][PC_STAGES][PC_STAGE]
  __shared__ uint64_t s_full[PC_WARPS][PC_STAGES];
  __shared__ PageTile s_tile[PC_WARPS][PC_STAGES];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < PC_WARPS * PC_STAGES) mbar_init(&s_full[0][0] + threadIdx.x, 1);
  fence_mbar_init();
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  if constexpr (REST) finish_compact(p);
  if (warp >= PC_WARPS) return;
  const int n = p.count ? *p.count : p.n;
  const long long all = (long long)n * p.n_layers * p.tiles, first = (long long)blockIdx.x * PC_WARPS + warp, step = (long long)gridDim.x * PC_WARPS;
  const int mine = first < all ? (int)((all - first + step - 1) / step) : 0;
  // lane i: tile base + i of this warp's
  PageTile ahead = {};
  auto look = [&](int base) {
    const int k = base + lane;
    ahead.tile = -1;
    if (k >= mine) return;
    const long long id = first + k * step, pl = id / p.tiles;
    const int i = (int)(pl / p.n_layers);
    ahead.layer = (int)(pl - (long long)i * p.n_layers);
    ahead.src = p.src[(size_t)i * p.step];
    ahead.dst = p.dst[(size_t)i * p.step];
    if ((unsigned)ahead.src >= (unsigned)p.c.n_pages || (unsigned)ahead.dst >= (unsigned)p.to_pages) raise_error(ERR_BAD_INPUT);
    else ahead.tile = (int)(id - pl * p.tiles);
  };
  auto load = [&](int k) {
    const int st = k % PC_STAGES;
    if (!(k & 31)) look(k);
    PageTile t;
    t.layer = __shfl_sync(0xffffffffu, ahead.layer, k & 31);
    t.src = __shfl_sync(0xffffffffu, ahead.src, k & 31);
    t.dst = __shfl_sync(0xffffffffu, ahead.dst, k & 31);
    t.tile = __shfl_sync(0xffffffffu, ahead.tile, k & 31);
    if (lane == 0) s_tile[warp][st] = t;
    const PagePiece x = page_piece<PC_STAGE>(p, t, lane);
    if (lane == 0) mbar_arrive_expect_tx(&s_full[warp][st], x.all);
    __syncwarp();
    if (x.bytes)
      bulk_load(s_stage + (warp * PC_STAGES + st) * PC_STAGE + x.at, page_array(p.from[t.layer], x.array) + x.from, x.bytes, &s_full[warp][st], l2_evict_first());
  };
  volatile int never = 0;
  bool ok = true;
  for (int k = 0; k < PC_LEAD && k < mine; ++k) load(k);
  for (int k = 0; k < mine && ok; ++k) {
    const int st = k % PC_STAGES;
    // the stage of the next tile to load was stored from PC_STAGES - PC_LEAD tiles ago
    if (k + PC_LEAD < mine) {
      bulk_wait_read<PC_STAGES - PC_LEAD - 1>();
      __syncwarp();
      load(k + PC_LEAD);
    }
    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s_full[warp][st], (k / PC_STAGES) & 1, &never));
    if (ok) {
      const PageTile t = s_tile[warp][st];
      const PagePiece x = page_piece<PC_STAGE>(p, t, lane);
      if (x.bytes) bulk_store(page_array(p.to[t.layer], x.array) + x.to, s_stage + (warp * PC_STAGES + st) * PC_STAGE + x.at, x.bytes);
    }
    bulk_commit();
  }
  bulk_wait_all();
  if (!ok) {                             // copies in flight get time to land
    raise_error(ERR_TIMEOUT_FULL);
    const unsigned long long w0 = global_ns();
    while (global_ns() - w0 < 50000ull) __nanosleep(1000);
  }
}

// ------------------------------------------------------------------ host side
static int check_pool(const sv_kv_pages* pages, PagePool* g) {
  if (!pages) return fail(SV_EINVAL, "pages must be non-null");
  if (!pages->refs || !pages->block_table || !pages->held || !aligned(pages->refs, 4) || !aligned(pages->block_table, 4) || !aligned(pages->held, 4))
    return fail(SV_EINVAL, "refs, block_table and held must be non-null and aligned");
  if (pages->page_size < 16 || pages->page_size > 65536 || (pages->page_size & (pages->page_size - 1)))
    return fail(SV_EUNSUPPORTED, "page_size must be a power of two in [16, 65536] (got %d)", pages->page_size);
  if (pages->n_pages < 1 || pages->n_pages > (1 << 30)) return fail(SV_EINVAL, "n_pages must be in [1, 2^30] (got %d)", pages->n_pages);
  if (pages->slots < 1 || pages->slots > MAX_BATCH) return fail(SV_EINVAL, "slots must be in [1, 256] (got %d)", pages->slots);
  g->refs = pages->refs;
  g->table = pages->block_table;
  g->held = pages->held;
  g->n_pages = pages->n_pages;
  g->page_shift = 0;
  while ((1 << g->page_shift) < pages->page_size) ++g->page_shift;
  g->slots = pages->slots;
  g->table_pages = pages->table_pages;
  if (pages->table_pages < 1) return fail(SV_EINVAL, "table_pages must be >= 1 (got %d)", pages->table_pages);
  if (((long long)pages->table_pages << g->page_shift) > (1ll << 30))
    return fail(SV_EUNSUPPORTED, "table_pages * page_size must be <= 2^30");
  if ((long long)pages->slots * pages->table_pages > (1ll << 30)) return fail(SV_EUNSUPPORTED, "slots * table_pages must be <= 2^30");
  return SV_OK;
}

// The layers' sizes into p; every layer is checked before anything is launched, and none is written twice.
static int check_layers(const sv_kv_cache* from, const sv_kv_cache* to, int n_layers, bool none, PageCopyParams* p) {
  if (n_layers < (none ? 0 : 1) || n_layers > 1024) return fail(SV_EINVAL, "n_layers must be in [%d, 1024] (got %d)", none ? 0 : 1, n_layers);
  if (n_layers && (!from || !to)) return fail(SV_EINVAL, "layers must be non-null");
  const void* seen[2 * 1024];
  for (int l = 0; l < n_layers; ++l) {
    KvCache a, b;
    int st = check_cache(from + l, &a);
    if (!st) st = check_cache(to + l, &b);
    if (st) return st;
    if (l == 0) {
      p->c = a;
      p->to_pages = b.n_pages;
    }
    if (a.page_shift != p->c.page_shift || a.heads != p->c.heads || a.dim != p->c.dim || a.bits != p->c.bits || a.n_pages != p->c.n_pages ||
        b.page_shift != a.page_shift || b.heads != a.heads || b.dim != a.dim || b.bits != a.bits || b.n_pages != p->to_pages)
      return fail(SV_EINVAL, "layer %d's cache differs in size or bits from layer 0's", l);
    seen[2 * l] = to[l].k;
    seen[2 * l + 1] = to[l].v;
  }
  std::sort(seen, seen + 2 * n_layers, std::less<const void*>());
  for (int i = 1; i < 2 * n_layers; ++i)
    if (seen[i] == seen[i - 1]) return fail(SV_EINVAL, "the same cache memory is listed twice");
  // one layer's copies may not write what another's read
  for (int l = 0; l < n_layers; ++l)
    for (const void* a : {from[l].k, from[l].v})
      if (a != to[l].k && a != to[l].v && std::binary_search(seen, seen + 2 * n_layers, a, std::less<const void*>()))
        return fail(SV_EINVAL, "layer %d is read from memory that another layer is written to", l);
  return SV_OK;
}

// REST: the first launch finishes a reserve (PART) or a compact too, and there is one even without layers.
template <bool PART, bool REST>
static cudaError_t launch_copy(const PageCopyParams& p, int grid, cudaStream_t s) {
  const auto kernel = PART ? kv_part_copy_kernel<REST> : p.stage == 8192 ? kv_page_copy_kernel<8192, REST> : kv_page_copy_kernel<16384, REST>;
  const int smem = PART ? 0 : PC_SMEM;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(grid), dim3(PC_THREADS), smem, s, attr);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
template <bool PART, bool REST>
static int launch_copies(PageCopyParams& p, const sv_kv_cache* from, const sv_kv_cache* to, int n_layers, cudaStream_t s) {
  const int sms = device_sm_count();
  if (sms <= 0) return fail(SV_ECUDA, "no CUDA device");
  const long long kv = n_layers ? (long long)p.c.heads * (p.c.dim * p.c.bits / 8) << p.c.page_shift : 0;   // bytes of an array's page
  const long long side = n_layers && p.c.bits != 16 ? (long long)p.c.heads * (p.c.dim / GROUP * 2) << p.c.page_shift : 0;
  auto tiles = [](long long bytes, long long size) { return (int)((bytes + size - 1) / size); };
  if (PART) {
    p.tiles_kv = tiles(kv, 16 * PP_TILE);
    p.tiles = 2 * p.tiles_kv + (side ? 1 : 0);
  } else {
    p.stage = kv < 16384 ? 8192 : 16384;
    p.tiles_kv = tiles(kv, p.stage);
    p.side_tiles = 4 * side <= p.stage ? 0 : tiles(side, p.stage);
    p.tiles = 2 * p.tiles_kv + (!side ? 0 : !p.side_tiles ? 1 : 4 * p.side_tiles);
  }
  for (int l0 = 0; l0 == 0 || l0 < n_layers; l0 += PG_LAYERS) {
    p.n_layers = n_layers - l0 < PG_LAYERS ? n_layers - l0 : PG_LAYERS;
    for (int l = 0; l < p.n_layers; ++l) {
      KvCache c;
      check_cache(from + l0 + l, &c);
      p.from[l] = c.p;
      check_cache(to + l0 + l, &c);
      p.to[l] = c.p;
    }
    const bool rest = REST && l0 == 0;
    const int each = PART ? 1 : PC_SMEM / (PC_STAGES * p.stage);
    long long want = ((long long)p.n * p.n_layers * p.tiles + each - 1) / each;
    if (rest && want < p.g.slots) want = p.g.slots;
    if (!want) continue;
    const int grid = (int)std::min(want, (long long)sms * (PART ? PP_CTAS : 1));
    const cudaError_t e = rest ? launch_copy<PART, REST>(p, grid, s) : launch_copy<PART, false>(p, grid, s);
    if (e != cudaSuccess) return cuda_fail(e, "page copy launch");
  }
  return SV_OK;
}

static size_t reserve_list_bytes(const PagePool& g) { return align256((size_t)g.n_pages * 4); }

}  // namespace sv

using namespace sv;

extern "C" {

int sv_kv_fork(const sv_kv_pages* pages, int n, const int32_t* parent, const int32_t* child, const int32_t* tokens, void* stream) {
  PagePool g;
  const int st = check_pool(pages, &g);
  if (st) return st;
  if (n < 0 || n > MAX_BATCH) return fail(SV_EINVAL, "n must be in [0, 256] (got %d)", n);
  if (!n) return SV_OK;
  if (!parent || !child || !tokens || !aligned(parent, 4) || !aligned(child, 4) || !aligned(tokens, 4))
    return fail(SV_EINVAL, "parent, child and tokens must be non-null and aligned");
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(n), dim3(128), 0, static_cast<cudaStream_t>(stream), attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_fork_kernel, g, n, parent, child, tokens);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "fork launch");
}

size_t sv_kv_reserve_workspace_bytes(const sv_kv_pages* pages) {
  PagePool g;
  return check_pool(pages, &g) ? 0 : reserve_list_bytes(g) + align256(MAX_BATCH * 4);
}

int sv_kv_reserve(const sv_kv_pages* pages, const sv_kv_cache* layers, int n_layers, const int32_t* keep, const int32_t* need,
                  int32_t* counts, int32_t* copies, void* workspace, size_t workspace_bytes, void* stream) {
  ReserveParams r;
  PageCopyParams p;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  int st = check_pool(pages, &r.g);
  if (!st) st = check_layers(layers, layers, n_layers, true, &p);
  if (st) return st;
  if (n_layers && (p.c.n_pages != r.g.n_pages || p.c.page_shift != r.g.page_shift))
    return fail(SV_EINVAL, "the caches' n_pages and page_size must be those of pages");
  if (!keep || !need || !counts || !copies || !aligned(keep, 4) || !aligned(need, 4) || !aligned(counts, 4) || !aligned(copies, 4))
    return fail(SV_EINVAL, "keep, need, counts and copies must be non-null and aligned");
  const size_t bytes = sv_kv_reserve_workspace_bytes(pages);
  if (!workspace || !aligned(workspace, 256)) return fail(SV_EINVAL, "workspace must be non-null and 256-byte aligned");
  if (workspace_bytes < bytes) return fail(SV_EINVAL, "workspace too small: %zu < %zu", workspace_bytes, bytes);
  r.keep = keep;
  r.need = need;
  r.counts = counts;
  r.copies = copies;
  r.list = static_cast<int32_t*>(workspace);
  r.before = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + reserve_list_bytes(r.g));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(1), dim3(PG_THREADS), 0, s, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_reserve_kernel, r);
  if (e != cudaSuccess) return cuda_fail(e, "reserve launch");
  p.g = r.g;
  p.list = r.list;
  p.before = r.before;
  p.fresh = counts + 2;
  p.src = copies;
  p.dst = copies + 1;
  p.places = copies + 2;
  p.step = 3;
  p.n = r.g.slots;
  p.count = counts + 1;
  return launch_copies<true, true>(p, layers, layers, n_layers, s);
}

int sv_kv_compact(const sv_kv_pages* pages, const sv_kv_cache* layers, int n_layers, int32_t* counts, int32_t* moves, void* stream) {
  PagePool g;
  PageCopyParams p;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  int st = check_pool(pages, &g);
  if (!st) st = check_layers(layers, layers, n_layers, true, &p);
  if (st) return st;
  if (n_layers && (p.c.n_pages != g.n_pages || p.c.page_shift != g.page_shift))
    return fail(SV_EINVAL, "the caches' n_pages and page_size must be those of pages");
  if (!counts || !moves || !aligned(counts, 4) || !aligned(moves, 4)) return fail(SV_EINVAL, "counts and moves must be non-null and aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(1), dim3(PG_THREADS), 0, s, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_compact_kernel, g, counts, moves);
  if (e != cudaSuccess) return cuda_fail(e, "compact launch");
  p.g = g;
  p.live = counts;
  p.src = moves;
  p.dst = moves + 1;
  p.step = 2;
  p.n = g.n_pages / 2;                   // a page that moves fills one that is free
  p.count = counts + 1;
  return launch_copies<false, true>(p, layers, layers, n_layers, s);
}

int sv_kv_copy_pages(const sv_kv_cache* from, const sv_kv_cache* to, int n_layers, int n, const int32_t* src, const int32_t* dst, void* stream) {
  PageCopyParams p;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  const int st = check_layers(from, to, n_layers, false, &p);
  if (st) return st;
  if (n < 0 || n > (1 << 24)) return fail(SV_EINVAL, "n must be in [0, 2^24] (got %d)", n);
  if (!n) return SV_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return fail(SV_EINVAL, "src and dst must be non-null and aligned");
  p.src = src;
  p.dst = dst;
  p.step = 1;
  p.n = n;
  return launch_copies<false, false>(p, from, to, n_layers, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
