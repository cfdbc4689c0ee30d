// Tree attention of a batch whose requests share prefixes: the entry point, and the join.
//
//   out = (sum over the prefix + sum over the request's own tokens) of p_t v_t / the same of p_t
//
// Softmax sums over parts of the tokens add up once they are brought to one maximum, so a prefix is attended to by all rows of its group
// at once (tree_attn_prefix.cu: its K and V are read once per 256 rows instead of once per request), and each request's own tokens
// by the kernels of tree attention, told to skip the prefix's pages.  Both leave fp32 sums with their maximum and weight; the join
// brings them together and rounds once.
//
// Measured (us, in a graph; 32 query and 8 key heads of 128, against tree attention of the same batch): 16 requests of 8 rows behind 16384
// tokens with up to 700 of their own, 8-bit, 81 to 86 against 169 (prefix 50, own tokens 25, join 8, less what overlaps); 64 of a row
// behind 8016 with up to 2011, 4-bit, 104 to 105 against 240 (30 to 40, 59, 14); 24 trees of up to 32 nodes in 48 heads behind 30000 and 25000,
// bf16, 273 to 279 against 478 (210, 56, 24).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "tree_attn_prefix.cuh"

namespace sv {

// Cached tokens times key heads that requests need not read again, from which on two more launches pay.  (8-bit, 32 query and 8 key heads,
// apart and together, us: 16 requests of a row over 1024 tokens 25.0 and 31.2, over 2048 31.2 and 34.5, over 4096 (491,520) 45.2 and 37.3, over
// 16384 119 and 47.5; 4 of 8 rows over 8192 35.3 and 41.4, over 16384 (393,216) 53.7 and 49.6, over 32768 94.6 and 76.2; other caches alike.
// One key head: 16 of 8 rows over 32768 (491,520) 53.6 and 59.8.  So two launches pay from 250 to 400 thousand on with eight key heads, and not
// yet at 490 thousand with one: the border is on the safe side, and leaves up to 8 us below it.)
constexpr double PX_WORTH = 500000.0;
// Of the plan's model, fitted to the times of such cases.  (PX_BEGIN 0 or 6: within 0.3 us in all of eight.  PX_PART 0: 16 x 1 row over 16384
// tokens 54.5 us instead of 48.3, 48 x 2 over 5000 57.6 instead of 59.6; 1: 64 x 1 over 8016 117 instead of 106, 4 x 8 over 32768 71 instead of
// 74.  PX_JOIN 0: 92.4 instead of 89.4 for 16 x 8 over 16384, 112 instead of 106 for 64 x 1; 1: 105 and 117, and 377 instead of 356 for 32 x 64
// over 2048.)
constexpr double PX_BEGIN = 3.0, PX_PART = 0.3, PX_JOIN = 0.3;
constexpr int TJ_WARPS = 8, TJ_CTAS = 4;       // warps a CTA, CTAs an SM
constexpr int TJ_AHEAD = 4;                    // parts of a row on their way at once

// One warp per (row, query head).  The parts of a row, in a fixed order: the prefix's, by tokens (two each where both matrices had the
// same rows), then the own tokens', by CTA.  A lane finds one part's place, maximum and weight, so that all parts' sums are asked for
// together, TJ_AHEAD at a time; what is read goes back to zero.  (A warp that went from part to part with all of its lanes: 44 us
// against 28 us for 396 rows of 48 heads in eight parts.)
template <int D>
__global__ void __launch_bounds__(32 * TJ_WARPS, TJ_CTAS) tree_attn_shared_join_kernel(const __grid_constant__ TreeAttnOwnParams p,
                                                                                       const __grid_constant__ PrefixParams x) {
  constexpr int E = D / 32;
  using Vec = std::conditional_t<E == 4, float4, float2>;
  __shared__ TaPlan plan;
  // what is looked up by request and group: indexed reads of the launch parameters take hundreds of cycles each
  __shared__ int s_offs[MAX_BATCH + 1];
  __shared__ short s_group[MAX_BATCH];
  __shared__ int s_rows[MAX_BATCH], s_row0[MAX_BATCH], s_pieces[MAX_BATCH], s_splits[MAX_BATCH], s_items[MAX_BATCH];
  const int lane = threadIdx.x & 31, B = p.map.B;
  if (threadIdx.x >= 32)
    for (int i = threadIdx.x - 32; i <= B; i += 32 * (TJ_WARPS - 1)) {
      s_offs[i] = p.map.offs[i];
      if (i < B) s_group[i] = x.group[i];
      if (i < x.n) {
        s_rows[i] = x.rows[i];
        s_row0[i] = x.row0[i];
        s_pieces[i] = x.pieces[i];
        s_splits[i] = x.splits[i];
        s_items[i] = x.items[i];
      }
    }
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 32) ta_plan(p, &plan, true, false);
  __syncthreads();
  const long long all = plan.pre[p.map.B], per = ta_div(all + p.grid - 1, p.grid);
  const unsigned heads = p.c.heads * p.group, units = p.map.offs[p.map.B] * heads;
  const int shift = 31 - __clz(p.block), x_all = x.pieces[x.n];   // (the block is a power of two)
  for (unsigned id = blockIdx.x * TJ_WARPS + (threadIdx.x >> 5); id < units; id += gridDim.x * TJ_WARPS) {
    const int row = (int)(id / heads), hq = (int)(id - row * heads), h = hq / p.group, hg = hq - h * p.group;
    int b = 0;
    for (int hi = B; hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if (s_offs[mid] <= row) b = mid; else hi = mid;
    }
    const int i = row - s_offs[b], m = s_offs[b + 1] - s_offs[b];
    // own tokens
    const int nt = (plan.len[b] + m + (1 << TA_UNIT_SHIFT) - 1) >> TA_UNIT_SHIFT, cost = ta_cost(p, m), r = i * p.group + hg;
    const int local = h * ta_blocks(m * p.group, p.block) + (r >> shift), k = r & (p.block - 1), item = (b ? plan.items[b] : 0) + local;
    const long long span = (long long)nt * cost, a0 = plan.pre[b] + (long long)local * (span + plan.begin);
    const int c0 = (int)ta_div(a0 + plan.begin + cost - 1, per), c1 = (int)ta_div(a0 + plan.begin + span - 1, per);
    // the prefix
    const int gi = s_group[b];
    int xn = 0, xrow = 0, xpiece = 0, halves = 0;
    if (gi >= 0) {
      const int xr = (row - s_row0[gi]) * p.group + hg, xrb = xr / PX_ROWS, xitem = h * px_blocks(s_rows[gi]) + xrb;
      xpiece = s_pieces[gi] + xitem * s_splits[gi];    // its first
      xrow = (s_items[gi] + xitem - xrb) * PX_ROWS + xr;
      halves = !px_pair(s_rows[gi], xrb);              // two parts a piece, as a shift
      xn = s_splits[gi] << halves;
    }
    const int n = xn + c1 - c0 + 1;
    float acc[E] = {}, weight = 0.f, most = -INFINITY;
    for (int j0 = 0; j0 < n; j0 += 32) {
      const int j = j0 + lane;
      unsigned place = 0;                              // row of the sums: in the prefix's, or the own tokens'
      float st = -INFINITY, wt = 0.f;
      float* at = nullptr;
      if (j < xn) {
        // a piece that another of its item and CTA comes before has no sums of its own
        const int piece = xpiece + (j >> halves), cta = px_cta(x_all, x.grid, piece);
        if (piece == xpiece || cta != px_cta(x_all, x.grid, piece - 1)) {
          place = xrow + cta * PX_ROWS + (halves ? (j & 1) * 128 : 0);
          at = x.stats + (size_t)place * TA_STAT;
        }
      } else if (j < n) {
        const int c = c0 + j - xn;
        const long long lo = (long long)c * per;
        if (ta_units_before(lo + per, a0, nt, cost, plan.begin) > ta_units_before(lo, a0, nt, cost, plan.begin)) {
          place = (item + c) * p.block + k;
          at = p.stats + (size_t)place * TA_STAT;
        }
      }
      if (at) {
        const float2 both = *reinterpret_cast<const float2*>(at);
        st = both.x;
        wt = both.y;
      }
      float top = fmaxf(most, st);
#pragma unroll
      for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float base = top == -INFINITY ? 0.f : top, fix = ta_exp2(most - base), w = ta_exp2(st - base);
      float sum = wt * w;
#pragma unroll
      for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      weight = weight * fix + sum;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= fix;
      most = top;
      unsigned parts = __ballot_sync(0xffffffffu, at != nullptr);
      while (parts) {
        Vec v[TJ_AHEAD];
        const unsigned now = parts;                    // the next TJ_AHEAD of them
#pragma unroll
        for (int y = 0; y < TJ_AHEAD; ++y) {
          const int src = parts ? __ffs(parts) - 1 : 0;
          const unsigned row_at = __shfl_sync(0xffffffffu, place, src);
          v[y] = Vec{};
          // (a part without weights may not have written its sums)
          if (parts && __shfl_sync(0xffffffffu, st, src) != -INFINITY)
            v[y] = reinterpret_cast<const Vec*>((j0 + src < xn ? x.partial : p.partial) + (size_t)row_at * D)[lane];
          parts &= parts - 1;
        }
        unsigned done = now;
#pragma unroll
        for (int y = 0; y < TJ_AHEAD; ++y) {
          const int src = done ? __ffs(done) - 1 : 0;
          const unsigned row_at = __shfl_sync(0xffffffffu, place, src);
          const float f = __shfl_sync(0xffffffffu, w, src);
          if (!done) break;
          acc[0] += v[y].x * f;
          acc[1] += v[y].y * f;
          if constexpr (E == 4) {
            acc[2] += v[y].z * f;
            acc[3] += v[y].w * f;
          }
          const bool pre = j0 + src < xn;
          reinterpret_cast<Vec*>((pre ? x.partial : p.partial) + (size_t)row_at * D)[lane] = Vec{};
          if (lane < 2) reinterpret_cast<float4*>((pre ? x.stats : p.stats) + (size_t)row_at * TA_STAT)[lane] = float4{};   // a whole sector
          done &= done - 1;
        }
      }
    }
    __nv_bfloat16* dst = p.out + (size_t)row * p.ldo + hq * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + e) =
          weight == 0.f ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(acc[e] / weight, acc[e + 1] / weight);
  }
}

// ------------------------------------------------------------------ host side
// Sizes of the sums, from the rows and the groups alone and never more for less of them, so that a workspace for the largest batch does
// for all: own tokens' as if blocks were the largest that the kernel of these rows takes, the prefixes' as if every group shared one.
struct SharedSizes {
  size_t partial, stats, px_partial, px_stats, total;
};
static int with_rows(const RowMap& map, const int32_t* group_offsets, int g) {
  int n = 0;
  for (int b = group_offsets[g]; b < group_offsets[g + 1]; ++b) n += map.offs[b + 1] > map.offs[b];
  return n;
}
static SharedSizes shared_sizes(const KvCache& c, const RowMap& map, int G, const int32_t* group_offsets, int heads_per) {
  int block;
  const int widest = ta_choose_block(map, heads_per, &block) ? 32 : 128;
  size_t own = ta_sms(), prefix = ta_sms();      // runs: one per item and CTA
  for (int b = 0; b < map.B; ++b) own += (size_t)c.heads * ta_blocks((map.offs[b + 1] - map.offs[b]) * heads_per, widest);
  for (int g = 0; g < G; ++g)
    if (with_rows(map, group_offsets, g) > 1)
      prefix += (size_t)c.heads * px_blocks((map.offs[group_offsets[g + 1]] - map.offs[group_offsets[g]]) * heads_per);
  SharedSizes z;
  z.partial = align256(own * widest * c.dim * sizeof(float));
  z.stats = align256(own * widest * TA_STAT * sizeof(float));
  z.px_partial = align256(prefix * PX_ROWS * c.dim * sizeof(float));
  z.px_stats = align256(prefix * PX_ROWS * TA_STAT * sizeof(float));
  z.total = std::max(ta_workspace_bytes(c), z.partial + z.stats + z.px_partial + z.px_stats);
  return z;
}

// What a call shares.  A group of one request has nothing to share: its prefix stays with the request, and so do all where there is
// little to save.
static int shared_plan(const KvCache& c, const RowMap& map, int G, const int32_t* group_offsets, const int32_t* shared_pages, int n_q_heads,
                       PrefixParams* x, int* skip) {
  if (G < 1 || G > MAX_BATCH) return fail(SV_EINVAL, "G must be in [1, 256] (got %d)", G);
  if (!group_offsets || !shared_pages) return fail(SV_EINVAL, "group_offsets and shared_pages must be non-null");
  if (group_offsets[0] != 0 || group_offsets[G] != map.B) return fail(SV_EINVAL, "group_offsets must go from 0 to B");
  for (int g = 0; g < G; ++g)
    if (group_offsets[g + 1] < group_offsets[g] || group_offsets[g + 1] > map.B) return fail(SV_EINVAL, "group_offsets must not decrease");
  for (int g = 0; g < G; ++g)
    if (shared_pages[g] < 0 || ((long long)shared_pages[g] << c.page_shift) > (1ll << 30))
      return fail(SV_EINVAL, "shared_pages[%d] must be in [0, 2^30 / page_size] (got %d)", g, shared_pages[g]);
  const int sms = ta_sms(), heads_per = n_q_heads / c.heads;
  x->heads_per = heads_per;
  x->n = 0;
  double saved = 0.0;
  auto alone = [&] {                     // every request attends to all of its tokens
    x->n = 0;
    for (int b = 0; b < map.B; ++b) {
      skip[b] = 0;
      x->group[b] = -1;
    }
  };
  alone();
  for (int g = 0; g < G; ++g) {
    const int requests = with_rows(map, group_offsets, g);
    if (requests < 2 || !shared_pages[g]) continue;
    int first = group_offsets[g];
    while (map.offs[first + 1] == map.offs[first]) ++first;
    saved += (double)(requests - 1) * ((long long)shared_pages[g] << c.page_shift) * c.heads;
    const int i = x->n++;
    x->row0[i] = map.offs[group_offsets[g]];
    x->rows[i] = (map.offs[group_offsets[g + 1]] - x->row0[i]) * heads_per;
    x->tokens[i] = shared_pages[g] << c.page_shift;
    x->request[i] = first;
    for (int b = group_offsets[g]; b < group_offsets[g + 1]; ++b) {
      skip[b] = shared_pages[g];
      x->group[b] = (short)i;
    }
  }
  if (saved < PX_WORTH) alone();
  if (!x->n) return SV_OK;
  // Pieces: of the numbers that come to up to twelve a CTA, the one that ends first, in tiles' time, where beginning and ending a run takes
  // as long as PX_BEGIN tiles, and the join of another part of every row PX_PART of them and PX_JOIN a thousand rows and query heads.
  auto cut = [&](double target) {        // tiles of a piece -> pieces
    int all = 0;
    x->pieces[0] = 0;
    for (int i = 0; i < x->n; ++i) {
      const int nt = px_tiles(x->tokens[i]), s = (int)(nt / target + 0.5);
      x->splits[i] = s < 1 ? 1 : (s > nt ? nt : s);
      all += c.heads * px_blocks(x->rows[i]) * x->splits[i];
      x->pieces[i + 1] = all;
    }
    return all;
  };
  double work = 0.0, rows = 0.0, best = 0.0, best_cost = 1e30;
  for (int i = 0; i < x->n; ++i) {
    work += (double)c.heads * px_blocks(x->rows[i]) * px_tiles(x->tokens[i]);
    rows += (double)c.heads * x->rows[i];
  }
  for (int each = -4; each <= 12; ++each)    // pieces a CTA, or (below 1) CTAs without one
    for (int less = 0; less < 2; ++less) {   // a little less than that many, or a little more
      const double many = each < 1 ? 0.5 / (1 << -each) : each, target = std::max(1.0, work / (many * sms) * (less ? 1.06 : 1.0));
      const int all = cut(target), most = (all + sms - 1) / sms;
      double longest = 0.0, parts = 0.0;
      for (int i = 0; i < x->n; ++i) {
        longest = std::max(longest, std::ceil((double)px_tiles(x->tokens[i]) / x->splits[i]));
        parts = std::max(parts, (1.0 + (double)(x->splits[i] - 1) / most) * (px_pair(x->rows[i], px_blocks(x->rows[i]) - 1) ? 1 : 2));
      }
      const double cost = most * longest + PX_BEGIN * (1.0 + (most - 1) / (double)x->splits[0]) + (PX_PART + PX_JOIN * 1e-3 * rows) * parts;
      if (cost < best_cost) {
        best_cost = cost;
        best = target;
      }
    }
  const int pieces = cut(best);
  x->grid = pieces < sms ? pieces : sms;
  for (int i = 0, items = 0; i < x->n; ++i) {
    x->items[i] = items;
    items += c.heads * px_blocks(x->rows[i]);
  }
  return SV_OK;
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_tree_attention_shared_workspace_bytes(const sv_kv_cache* cache, int G, const int32_t* group_offsets, const int32_t* shared_pages,
                                                int B, const int32_t* row_offsets, int n_q_heads) {
  KvCache c;
  RowMap m;
  PrefixParams x;
  int skip[MAX_BATCH];
  if (ta_check_batch(cache, B, row_offsets, n_q_heads, &c, &m) || shared_plan(c, m, G, group_offsets, shared_pages, n_q_heads, &x, skip)) return 0;
  return shared_sizes(c, m, G, group_offsets, n_q_heads / c.heads).total;
}

int sv_tree_attention_shared(const sv_kv_cache* cache, int G, const int32_t* group_offsets, const int32_t* shared_pages, int B,
                             const int32_t* row_offsets, const int32_t* kv_len, const int32_t* block_table, int table_pages,
                             const uint16_t* q, int ldq, int n_q_heads, float scale, const uint64_t* tree_mask, uint16_t* out, int ldo,
                             void* workspace, size_t workspace_bytes, void* stream) {
  TreeAttnOwnParams p;
  PrefixParams x;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  memset(static_cast<void*>(&x), 0, sizeof(x));
  int st = ta_check_batch(cache, B, row_offsets, n_q_heads, &p.c, &p.map);
  if (!st) st = ta_check_call(&p, kv_len, block_table, table_pages, q, ldq, n_q_heads, scale, tree_mask, out, ldo);
  if (!st) st = shared_plan(p.c, p.map, G, group_offsets, shared_pages, n_q_heads, &x, p.skip);
  if (st) return st;
  for (int g = 0; g < G; ++g)
    if (shared_pages[g] > table_pages) return fail(SV_EINVAL, "shared_pages[%d] is more than table_pages", g);
  if (!workspace || !aligned(workspace, 256)) return fail(SV_EINVAL, "workspace must be non-null and 256-byte aligned");
  const SharedSizes z = shared_sizes(p.c, p.map, G, group_offsets, x.heads_per);
  const size_t bytes = x.n ? z.total : ta_workspace_bytes(p.c);
  if (workspace_bytes < bytes) return fail(SV_EINVAL, "workspace too small: %zu < %zu", workspace_bytes, bytes);
  if (!x.n)                               // nothing is shared
    return sv_tree_attention(cache, B, row_offsets, kv_len, block_table, table_pages, q, ldq, n_q_heads, scale, tree_mask, out, ldo, workspace,
                             workspace_bytes, stream);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.partial = reinterpret_cast<float*>(ws);
  p.stats = reinterpret_cast<float*>(ws + z.partial);
  x.partial = reinterpret_cast<float*>(ws + z.partial + z.stats);
  x.stats = reinterpret_cast<float*>(ws + z.partial + z.stats + z.px_partial);
  x.c = p.c;
  x.table = block_table;
  x.table_pages = table_pages;
  x.q = p.q;
  x.ldq = ldq;
  x.scale = scale;
  for (int b = 0; b < B; ++b)             // before the first launch
    if (((long long)(table_pages - p.skip[b]) << p.c.page_shift) < p.map.offs[b + 1] - p.map.offs[b])
      return fail(SV_EINVAL, "request %d has more rows than block_table has places", b);
  if (p.c.bits == 16) {
    st = ta_encode(p.c, &x.tk, &x.tv);
    if (st) return st;
  }
  cudaError_t e = launch_tree_attn_prefix(x, s);
  if (e != cudaSuccess) return cuda_fail(e, "prefix attention launch");
  bool one_unit;
  st = ta_launch(&p, s, &one_unit);
  if (st) return st;
  const long long units = (long long)p.map.offs[B] * n_q_heads, ctas = (units + TJ_WARPS - 1) / TJ_WARPS, most = (long long)TJ_CTAS * ta_sms();
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)(ctas < most ? ctas : most)), dim3(32 * TJ_WARPS), 0, s, attr);
  e = p.c.dim == 128 ? cudaLaunchKernelEx(&cfg, tree_attn_shared_join_kernel<128>, p, x) : cudaLaunchKernelEx(&cfg, tree_attn_shared_join_kernel<64>, p, x);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "prefix join launch");
}

}  // extern "C"
