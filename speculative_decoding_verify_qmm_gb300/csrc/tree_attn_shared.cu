// Tree attention of a batch whose requests share prefixes: the entry point, and the join.
//
//   out = (sum over the prefix + sum over the request's own tokens) of p_t v_t / the same of p_t
//
// Softmax sums over parts of the tokens add up once they are brought to one maximum, so a prefix is attended to by all rows of its group
// at once (tree_attn_prefix.cu: its K and V are read once per 256 rows instead of once per request), and each request's own tokens
// by the kernels of tree attention, told to skip the prefix's pages.  Both leave fp32 sums with their maximum and weight; the join
// brings them together and rounds once.
#include <cstring>

#include "tree_attn_prefix.cuh"

namespace sv {

constexpr int TJ_WARPS = 8, TJ_AHEAD = 4;      // warps a CTA, parts of a row on their way at once

// One warp per (row, query head).  The parts of a row, in a fixed order: the prefix's, by CTA (two each where both matrices had the
// same rows), then the own tokens', by CTA.  What is read goes back to zero.
template <int D>
__global__ void __launch_bounds__(32 * TJ_WARPS) tree_attn_shared_join_kernel(const __grid_constant__ TreeAttnParams p,
                                                                              const __grid_constant__ PrefixParams x) {
  constexpr int E = D / 32;
  __shared__ TaPlan plan;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 32) ta_plan(p, &plan, true, false);
  __syncthreads();
  const long long all = plan.pre[p.map.B], per = ta_div(all + p.grid - 1, p.grid);
  const int heads = p.c.heads * p.group;
  const long long pairs = (long long)p.map.offs[p.map.B] * heads;
  for (long long id = (long long)blockIdx.x * TJ_WARPS + (threadIdx.x >> 5); id < pairs; id += (long long)gridDim.x * TJ_WARPS) {
    const int row = (int)ta_div(id, heads), hq = (int)(id - (long long)row * heads), h = hq / p.group;
    const int b = request_of(p.map, row), i = row - p.map.offs[b], m = p.map.offs[b + 1] - p.map.offs[b];
    // the own tokens' parts
    const int r = i * p.group + (hq - h * p.group), rb = r / p.block, k = r - rb * p.block;
    const int nt = (plan.len[b] + m + (1 << TA_UNIT_SHIFT) - 1) >> TA_UNIT_SHIFT, cost = ta_cost(p, m);
    const long long span = (long long)nt * cost;
    const int local = h * ta_blocks(m * p.group, p.block) + rb, item = (b ? plan.items[b] : 0) + local;
    const long long a0 = plan.pre[b] + (long long)local * (span + plan.begin);
    const int c0 = (int)ta_div(a0 + plan.begin + cost - 1, per), c1 = (int)ta_div(a0 + plan.begin + span - 1, per);
    // the prefix's
    const int gi = x.group[b];
    int xc0 = 0, xn = 0, xk = 0, xitem = 0, xcost = 1, xnt = 0, halves = 1;
    long long xa0 = 0;
    if (gi >= 0) {
      const PxGroup g = px_group(x, x.rows[gi], x.tokens[gi]);
      const int xr = (row - x.row0[gi]) * p.group + (hq - h * p.group), xrb = xr / PX_ROWS;
      xk = xr - xrb * PX_ROWS;
      const bool pair = xrb < g.blocks - 1 || g.last;
      xcost = x.cost[pair];
      xnt = g.nt;
      xa0 = x.pre[gi] + h * g.span + xrb * g.full;
      xitem = x.items[gi] + h * g.blocks + xrb;
      halves = pair ? 1 : 2;
      xc0 = (int)ta_div(xa0 + x.begin_cost + xcost - 1, x.per);
      xn = ((int)ta_div(xa0 + x.begin_cost + (long long)xnt * xcost - 1, x.per) - xc0 + 1) * halves;
    }
    const int n = xn + c1 - c0 + 1;
    float acc[E] = {}, weight = 0.f, most = -INFINITY;
    for (int j0 = 0; j0 < n; j0 += TJ_AHEAD) {
      float *sums[TJ_AHEAD], *stat[TJ_AHEAD];
      int step[TJ_AHEAD];
      float st[TJ_AHEAD], wt[TJ_AHEAD], v[TJ_AHEAD][E];
#pragma unroll
      for (int y = 0; y < TJ_AHEAD; ++y) {
        const int j = j0 + y;
        sums[y] = nullptr;
        if (j < xn) {
          const int c = xc0 + j / halves;
          const long long lo = (long long)c * x.per;
          if (ta_units_before(lo + x.per, xa0, xnt, xcost, x.begin_cost) > ta_units_before(lo, xa0, xnt, xcost, x.begin_cost)) {
            const size_t slot = (size_t)xitem + c;
            const int kk = xk + (halves == 2 ? (j & 1) * 128 : 0);
            sums[y] = x.partial + (slot * PX_ROWS + kk) * D;
            stat[y] = x.stats + slot * (2 * PX_ROWS) + kk;
            step[y] = PX_ROWS;
          }
        } else if (j < n) {
          const int c = c0 + j - xn;
          const long long lo = (long long)c * per;
          if (ta_units_before(lo + per, a0, nt, cost, plan.begin) > ta_units_before(lo, a0, nt, cost, plan.begin)) {
            const size_t slot = (size_t)item + c;
            sums[y] = p.partial + (slot * p.block + k) * D;
            stat[y] = p.stats + 2 * slot * p.block + k;
            step[y] = p.block;
          }
        }
        st[y] = -INFINITY;
        wt[y] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[y][e] = 0.f;
        if (sums[y]) {
          st[y] = stat[y][0];
          wt[y] = stat[y][step[y]];
          if constexpr (E == 4) {
            const float4 t = reinterpret_cast<const float4*>(sums[y])[lane];
            v[y][0] = t.x; v[y][1] = t.y; v[y][2] = t.z; v[y][3] = t.w;
          } else {
            const float2 t = reinterpret_cast<const float2*>(sums[y])[lane];
            v[y][0] = t.x; v[y][1] = t.y;
          }
        }
      }
      __syncwarp();                      // every lane has the statistics
      float top = most;
#pragma unroll
      for (int y = 0; y < TJ_AHEAD; ++y) {
        top = fmaxf(top, st[y]);
        if (!sums[y]) continue;
        if constexpr (E == 4) reinterpret_cast<float4*>(sums[y])[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
        else reinterpret_cast<float2*>(sums[y])[lane] = make_float2(0.f, 0.f);
        if (lane < 2) stat[y][lane * step[y]] = 0.f;
      }
      const float base = top == -INFINITY ? 0.f : top, fix = ta_exp2(most - base);
      weight *= fix;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= fix;
#pragma unroll
      for (int y = 0; y < TJ_AHEAD; ++y) {
        const float w = ta_exp2(st[y] - base);
        weight += wt[y] * w;
        // a part without weights may not have written its sums
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += st[y] == -INFINITY ? 0.f : v[y][e] * w;
      }
      most = top;
    }
    __nv_bfloat16* dst = p.out + (size_t)row * p.ldo + hq * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + e) =
          weight == 0.f ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(acc[e] / weight, acc[e + 1] / weight);
  }
}

// ------------------------------------------------------------------ host side
// What a call shares: the groups whose prefix is worth a pass of its own, and the sizes of the sums.  A group of one request has nothing
// to share: its prefix stays with the request.
struct SharedSizes {
  size_t partial, stats, px_partial, px_stats, total;
};
static int shared_plan(const KvCache& c, const RowMap& map, int G, const int32_t* group_offsets, const int32_t* shared_pages, int n_q_heads,
                       PrefixParams* x, int* skip, SharedSizes* z) {
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
  x->cost[0] = 6;
  x->cost[1] = 10;
  x->begin_cost = 40;
  x->n = 0;
  for (int b = 0; b < map.B; ++b) {
    skip[b] = 0;
    x->group[b] = -1;
  }
  long long items = 0;
  for (int g = 0; g < G; ++g) {
    int first = -1, with_rows = 0;
    for (int b = group_offsets[g]; b < group_offsets[g + 1]; ++b)
      if (map.offs[b + 1] > map.offs[b]) {
        if (first < 0) first = b;
        ++with_rows;
      }
    if (with_rows < 2 || !shared_pages[g]) continue;
    const int i = x->n++;
    x->row0[i] = map.offs[group_offsets[g]];
    x->rows[i] = (map.offs[group_offsets[g + 1]] - x->row0[i]) * heads_per;
    x->tokens[i] = shared_pages[g] << c.page_shift;
    x->request[i] = first;
    const PxGroup s = px_group(*x, x->rows[i], x->tokens[i]);
    x->pre[i + 1] = x->pre[i] + c.heads * s.span;
    items += (long long)c.heads * s.blocks;
    x->items[i + 1] = (int)items;
    for (int b = group_offsets[g]; b < group_offsets[g + 1]; ++b) {
      skip[b] = shared_pages[g];
      x->group[b] = (short)i;
    }
  }
  memset(z, 0, sizeof(*z));
  z->total = ta_workspace_bytes(c);
  if (!x->n) return SV_OK;
  x->grid = x->pre[x->n] < sms ? (int)x->pre[x->n] : sms;
  x->per = (x->pre[x->n] + x->grid - 1) / x->grid;
  int block;
  ta_choose_block(map, heads_per, &block);
  size_t own = sms;                              // runs of own tokens: one per item and CTA
  for (int b = 0; b < map.B; ++b) own += (size_t)c.heads * ta_blocks((map.offs[b + 1] - map.offs[b]) * heads_per, block);
  z->partial = align256(own * block * c.dim * sizeof(float));
  z->stats = align256(own * block * 2 * sizeof(float));
  z->px_partial = align256((items + sms) * PX_ROWS * c.dim * sizeof(float));
  z->px_stats = align256((items + sms) * PX_ROWS * 2 * sizeof(float));
  const size_t need = z->partial + z->stats + z->px_partial + z->px_stats;
  if (need > z->total) z->total = need;
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
  SharedSizes z;
  x.pre[0] = 0;
  x.items[0] = 0;
  if (ta_check_batch(cache, B, row_offsets, n_q_heads, &c, &m) || shared_plan(c, m, G, group_offsets, shared_pages, n_q_heads, &x, skip, &z)) return 0;
  return z.total;
}

int sv_tree_attention_shared(const sv_kv_cache* cache, int G, const int32_t* group_offsets, const int32_t* shared_pages, int B,
                             const int32_t* row_offsets, const int32_t* kv_len, const int32_t* block_table, int table_pages,
                             const uint16_t* q, int ldq, int n_q_heads, float scale, const uint64_t* tree_mask, uint16_t* out, int ldo,
                             void* workspace, size_t workspace_bytes, void* stream) {
  TreeAttnParams p;
  PrefixParams x;
  SharedSizes z;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  memset(static_cast<void*>(&x), 0, sizeof(x));
  int st = ta_check_batch(cache, B, row_offsets, n_q_heads, &p.c, &p.map);
  if (!st) st = ta_check_call(&p, kv_len, block_table, table_pages, q, ldq, n_q_heads, scale, tree_mask, out, ldo);
  if (!st) st = shared_plan(p.c, p.map, G, group_offsets, shared_pages, n_q_heads, &x, p.skip, &z);
  if (st) return st;
  for (int g = 0; g < G; ++g)
    if (shared_pages[g] > table_pages) return fail(SV_EINVAL, "shared_pages[%d] is more than table_pages", g);
  if (!workspace || !aligned(workspace, 256)) return fail(SV_EINVAL, "workspace must be non-null and 256-byte aligned");
  if (workspace_bytes < z.total) return fail(SV_EINVAL, "workspace too small: %zu < %zu", workspace_bytes, z.total);
  if (!x.n)                               // nothing is shared
    return sv_tree_attention(cache, B, row_offsets, kv_len, block_table, table_pages, q, ldq, n_q_heads, scale, tree_mask, out, ldo, workspace,
                             workspace_bytes, stream);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.partial = reinterpret_cast<float*>(ws);
  p.stats = reinterpret_cast<float*>(ws + z.partial);
  p.keep = 1;
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
  const long long pairs = (long long)p.map.offs[B] * n_q_heads, ctas = (pairs + TJ_WARPS - 1) / TJ_WARPS, most = 8ll * ta_sms();
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)(ctas < most ? ctas : most)), dim3(32 * TJ_WARPS), 0, s, attr);
  e = p.c.dim == 128 ? cudaLaunchKernelEx(&cfg, tree_attn_shared_join_kernel<128>, p, x) : cudaLaunchKernelEx(&cfg, tree_attn_shared_join_kernel<64>, p, x);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "prefix join launch");
}

}  // extern "C"
