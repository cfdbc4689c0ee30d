// Attention of the drafted rows over the paged cache: the entry point, and the join of items that spanned CTAs (the kernel
// itself is tree_attn_narrow.cuh up to 32 rows and tree_attn_wide.cu above).
#include <cmath>
#include <cstddef>
#include <cstring>

#include "tree_attn.cuh"

namespace sv {

// Up to 32 rows a key head the warp-level kernel, above the tensor-memory one.  48 rows (4 requests of 8 rows in 48 heads, 30001
// tokens, 8-bit): 113 us against 54.  32 rows (8 rows, 32 heads, 8-bit): 14.9 us against 15.2 at 2048 tokens, 16.3 against 23.0 at 8192,
// 23.2 against 21.4 at 16384, 52 against 43 at 65536; 20 rows, 4-bit and bf16 caches alike (bf16: 17.7 and 21.8 at 8192, 54 and 52 at
// 65536).  Lengths are on the device, so the better one for short contexts has them all.
constexpr int TA_MAX_BLOCK = 128, TA_NARROW_ROWS = 32;

// Joins the partial sums of items that spanned CTAs, in CTA order.  WPP warps per (row, query head) take every WPP-th part,
// eight parts on their way at once, and meet in shared memory in warp order.  PAIRS such pairs a CTA at a time.  All that
// does not read the parts is done before the wait for them.  A part is read once, and its place left at zero, as other calls
// that use the same workspace expect (0.5 to 2.5 us, where the calls that need zeros would otherwise need a workspace of their own).
// Bound by latency: some 2 us behind the last part for one to 32 rows, 4 to 5 us for the largest (12 MB read and zeroed).
template <int D, int WPP, int PAIRS>
__global__ void __launch_bounds__(32 * WPP * PAIRS) tree_attn_join_kernel(const __grid_constant__ TreeAttnParams p) {
  constexpr int E = D / 32;
  __shared__ TaPlan plan;
  __shared__ float s_acc[PAIRS][WPP][WPP > 1 ? D : 1], s_most[PAIRS][WPP], s_weight[PAIRS][WPP];
  const int lane = threadIdx.x & 31, pair = (threadIdx.x >> 5) / WPP, warp = (threadIdx.x >> 5) % WPP;
  // The kernel before lets this one start only after its own wait, so what came before it is there already.
  if (threadIdx.x < 32) ta_plan(p, &plan, true, false);
  __syncthreads();
  const long long all = plan.pre[p.map.B], per = ta_div(all + p.grid - 1, p.grid);
  const int heads = p.c.heads * p.group;
  const long long pairs = (long long)p.map.offs[p.map.B] * heads;
  int row, hq, k, c0, c1, nt, cost;
  long long a0;
  auto locate = [&](long long id) {
    row = (int)ta_div(id, heads);
    hq = (int)(id - (long long)row * heads);
    const int b = request_of(p.map, row), i = row - p.map.offs[b], m = p.map.offs[b + 1] - p.map.offs[b];
    const int h = hq / p.group, r = i * p.group + (hq - h * p.group), rb = r / p.block;
    k = r - rb * p.block;
    nt = (plan.len[b] + m + (1 << TA_UNIT_SHIFT) - 1) >> TA_UNIT_SHIFT;
    cost = ta_cost(p, m);
    const long long span = (long long)nt * cost;
    a0 = plan.pre[b] + ((long long)h * ta_blocks(m * p.group, p.block) + rb) * (span + plan.begin);
    // the first and the last CTA with units of this item (one between them may have none where shares are small)
    c0 = (int)ta_div(a0 + plan.begin + cost - 1, per);
    c1 = (int)ta_div(a0 + plan.begin + span - 1, per);
  };
  const long long first = (long long)blockIdx.x * PAIRS + pair, step = (long long)gridDim.x * PAIRS;
  if (first < pairs) locate(first);                    // before the wait: all that does not read the parts
  const bool dense = per >= 12;                        // more than any unit costs: every CTA of a share has units
  pdl_wait();
  pdl_trigger();
  for (long long id = first; id < pairs; id += step) {
    if (id != first) locate(id);
    if (c0 == c1) continue;                            // one CTA had the whole item and wrote the output
    float acc[E] = {}, weight = 0.f, most = -INFINITY;
    for (int c8 = c0 + warp; c8 <= c1; c8 += 8 * WPP) {
      float x[8][E], st[8], wt[8];
      int from[8];                                     // the part's slot; -1: none
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const int c = c8 + WPP * y;
        const long long lo = (long long)c * per;
        from[y] = -1;
        st[y] = -INFINITY;
        wt[y] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x[y][e] = 0.f;
        if (c <= c1 && (dense || ta_units_before(lo + per, a0, nt, cost, plan.begin) > ta_units_before(lo, a0, nt, cost, plan.begin))) {
          const size_t slot = 2 * (size_t)c + (a0 > lo ? 1 : 0);   // the CTA's first item if its share begins in it
          from[y] = (int)slot;
          st[y] = p.stats[2 * slot * p.block + k];
          wt[y] = p.stats[(2 * slot + 1) * p.block + k];
          const float* src = p.partial + (slot * p.block + k) * D + lane * E;
          if constexpr (E == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            x[y][0] = v.x; x[y][1] = v.y; x[y][2] = v.z; x[y][3] = v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            x[y][0] = v.x; x[y][1] = v.y;
          }
        }
      }
      __syncwarp();                                    // every lane has the statistics: what was read goes back to zero
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        if (from[y] < 0) continue;
        const size_t at = (size_t)from[y];
        float* src = p.partial + (at * p.block + k) * D + lane * E;
        if constexpr (E == 4) *reinterpret_cast<float4*>(src) = make_float4(0.f, 0.f, 0.f, 0.f);
        else *reinterpret_cast<float2*>(src) = make_float2(0.f, 0.f);
        if (lane < 2) p.stats[(2 * at + lane) * p.block + k] = 0.f;
      }
      float top = most;
#pragma unroll
      for (int y = 0; y < 8; ++y) top = fmaxf(top, st[y]);
      const float base = top == -INFINITY ? 0.f : top, fix = ta_exp2(most - base);
      weight *= fix;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= fix;
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const float w = ta_exp2(st[y] - base);
        weight += wt[y] * w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += x[y][e] * w;
      }
      most = top;
    }
    if constexpr (WPP > 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) s_acc[pair][warp][lane * E + e] = acc[e];
      if (lane == 0) {
        s_most[pair][warp] = most;
        s_weight[pair][warp] = weight;
      }
      named_bar_sync(1 + pair, 32 * WPP);
      for (int w = 0; w < WPP; ++w) most = fmaxf(most, s_most[pair][w]);
      const float base = most == -INFINITY ? 0.f : most;
      float f[WPP];
      weight = 0.f;
#pragma unroll
      for (int w = 0; w < WPP; ++w) {
        f[w] = ta_exp2(s_most[pair][w] - base);
        weight += s_weight[pair][w] * f[w];
      }
      for (int d = 32 * warp + lane; d < D; d += 32 * WPP) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < WPP; ++w) sum += s_acc[pair][w][d] * f[w];
        p.out[(size_t)row * p.ldo + hq * D + d] = __float2bfloat16_rn(weight == 0.f ? 0.f : sum / weight);
      }
      if (gridDim.x * PAIRS < pairs) named_bar_sync(1 + pair, 32 * WPP);   // another round follows
      continue;
    }
    __nv_bfloat16* dst = p.out + (size_t)row * p.ldo + hq * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + e) =
          weight == 0.f ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(acc[e] / weight, acc[e + 1] / weight);
  }
}

// ------------------------------------------------------------------ host side
static int check_heads(const KvCache& c, int n_q_heads) {
  if (c.dim != 64 && c.dim != 128) return fail(SV_EUNSUPPORTED, "attention needs head_dim 64 or 128 (got %d)", c.dim);
  if (n_q_heads < c.heads || n_q_heads % c.heads || n_q_heads / c.heads > 64)
    return fail(SV_EINVAL, "n_q_heads must be 1 to 64 times n_kv_heads (got %d, %d)", n_q_heads, c.heads);
  if ((long long)c.n_pages * c.heads > 0x7fffffffll) return fail(SV_EUNSUPPORTED, "n_pages * n_kv_heads must be below 2^31");
  return SV_OK;
}

int ta_check_batch(const sv_kv_cache* cache, int B, const int32_t* row_offsets, int n_q_heads, KvCache* c, RowMap* m) {
  int st = check_cache(cache, c);
  if (!st) st = check_rows_map(B, row_offsets, KV_MAX_DRAFT, 1 << 22, m);
  return st ? st : check_heads(*c, n_q_heads);
}

// One CTA per SM (152 where no device is present: sizes only).
int ta_sms() {
  const int n = device_sm_count();
  return n > 0 ? n : 152;
}
static size_t ta_partial_bytes(int grid, int dim) { return (size_t)2 * grid * TA_MAX_BLOCK * dim * sizeof(float); }
static size_t ta_stats_bytes(int grid) { return (size_t)4 * grid * TA_MAX_BLOCK * sizeof(float); }
size_t ta_workspace_bytes(const KvCache& c) { return ta_partial_bytes(ta_sms(), c.dim) + ta_stats_bytes(ta_sms()); }

bool ta_choose_block(const RowMap& map, int group, int* block) {
  int rows = 0;                // of the widest request, times the group
  long long by16 = 0, by32 = 0;
  for (int b = 0; b < map.B; ++b) {
    const int m = map.offs[b + 1] - map.offs[b];
    if (m * group > rows) rows = m * group;
    by16 += 4 * ta_blocks(m * group, 16);
    by32 += m ? (m * group > 16 ? 7 : 5) : 0;
  }
  const bool narrow = rows <= TA_NARROW_ROWS;
  // In fifths of the time of a narrow unit of 32-row blocks with one row tile filled: two tiles filled take 7, a block of 16
  // rows takes 4.  (One request of 32 rows over 16384 tokens: 23.3 us in a block of 32, 23.8 in two of 16, over 65536 52 and 61; 48
  // requests of 4 to 20 rows: 191 in blocks of 32, 158 in blocks of 16.)
  *block = narrow ? (by16 < by32 ? 16 : 32) : TA_MAX_BLOCK;
  return narrow;
}

int ta_check_call(TreeAttnParams* out, const int32_t* kv_len, const int32_t* block_table, int table_pages, const uint16_t* q, int ldq,
                  int n_q_heads, float scale, const uint64_t* tree_mask, uint16_t* to, int ldo) {
  TreeAttnParams& p = *out;
  const int st = check_table(p.c, kv_len, block_table, table_pages);
  if (st) return st;
  if (!q || !to || !aligned(q, 16) || !aligned(to, 16) || ldq % 8 || ldo % 8)
    return fail(SV_EINVAL, "q and out must be non-null, 16-byte aligned, with strides that are multiples of 8");
  if (ldq < n_q_heads * p.c.dim || ldo < n_q_heads * p.c.dim) return fail(SV_EINVAL, "ldq and ldo must be >= n_q_heads * head_dim");
  if (q == to && ldq != ldo && p.map.offs[p.map.B] > 1) return fail(SV_EINVAL, "an in-place call needs equal strides");
  if (!(std::fabs(scale) <= 0x1p127f)) return fail(SV_EINVAL, "scale must be at most 2^127 in magnitude");
  if (!aligned(tree_mask, 8)) return fail(SV_EINVAL, "tree_mask must be 8-byte aligned");
  p.kv_len = kv_len;
  p.table = block_table;
  p.table_pages = table_pages;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.ldq = ldq;
  p.group = n_q_heads / p.c.heads;
  p.per_group = ((1u << 20) + p.group - 1) / p.group;
  p.scale = scale;
  p.mask = tree_mask;
  p.out = reinterpret_cast<__nv_bfloat16*>(to);
  p.ldo = ldo;
  return SV_OK;
}

int ta_encode(const KvCache& c, CUtensorMap* tk, CUtensorMap* tv) {
  const uint64_t slabs = (uint64_t)c.n_pages * c.heads, page = 1ull << c.page_shift;
  const uint32_t box = page < 128 ? (uint32_t)page : 128u;
  const int st = encode_tiled_3d_sw128(tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, c.p.k, c.dim, page, slabs, 2, 64, box);
  return st ? st : encode_tiled_3d_sw128(tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, c.p.v, c.dim, page, slabs, 2, 64, box);
}

template <typename P>
int ta_launch(P* out, cudaStream_t s, bool* one_unit) {
  P& p = *out;
  const bool narrow = ta_choose_block(p.map, p.group, &p.block);
  // Beginning an item, in the same measure: what gave the least time over several batches and lengths.  (Wide, bf16, 32 rows of
  // 65536 tokens: 60.8 us with 30, 59.0 with 60; 4 x 8 rows in 48 heads 68.0 and 64.2, over codes 54.8 and 56.1.  Narrow, 8-bit,
  // 8 rows of 65536 tokens: 57.4 with 25, 52.8 with 35; 8 x 4 rows 32.4 and 33.2.)
  p.cost[0] = 5;
  p.cost[1] = p.block == 32 ? 7 : 5;
  p.begin_cost = narrow ? (p.block == 16 ? 25 : 35) : (p.c.bits == 16 ? 60 : 35);
  // the lengths are on the device: size the grid for the longest the table allows
  long long most = 0;
  *one_unit = true;
  for (int b = 0; b < p.map.B; ++b) {
    const int m = p.map.offs[b + 1] - p.map.offs[b];
    const long long places = (long long)(p.table_pages - ta_skip(p, b)) << p.c.page_shift;
    if (m > places) return fail(SV_EINVAL, "request %d has more rows than block_table has places", b);
    const long long units = (places + (1 << TA_UNIT_SHIFT) - 1) >> TA_UNIT_SHIFT;
    most += (long long)p.c.heads * ta_blocks(m * p.group, p.block) * units;
    if (m && units > 1) *one_unit = false;
  }
  const int sms = ta_sms();
  p.grid = most < sms ? (int)most : sms;
  if (p.c.bits == 16 && !narrow) {
    const int st = ta_encode(p.c, &p.tk, &p.tv);
    if (st) return st;
  }
  const cudaError_t e = narrow ? launch_tree_attn_narrow(p, s) : launch_tree_attn_wide(p, s);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "tree attention launch");
}
template int ta_launch(TreeAttnParams*, cudaStream_t, bool*);
template int ta_launch(TreeAttnOwnParams*, cudaStream_t, bool*);

template <int D, int WPP, int PAIRS>
static cudaError_t launch_join_w(const TreeAttnParams& p, long long pairs, long long most, cudaStream_t s) {
  const long long ctas = (pairs + PAIRS - 1) / PAIRS;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)(ctas < most ? ctas : most)), dim3(32 * WPP * PAIRS), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, tree_attn_join_kernel<D, WPP, PAIRS>, p);
}
// Few pairs: a small CTA each, all there at once (0.8 us from the last part to the output, against 2.4 with the large
// ones).  Many: one large CTA per SM, which comes in as the kernel before leaves the SM; CTA after CTA would come in too late.
template <int D>
static cudaError_t launch_join(const TreeAttnParams& p, int sms, cudaStream_t s) {
  const long long pairs = (long long)p.map.offs[p.map.B] * p.c.heads * p.group;
  if (pairs <= 4ll * sms) return launch_join_w<D, 4, 1>(p, pairs, pairs, s);
  return pairs <= 8ll * sms ? launch_join_w<D, 2, 8>(p, pairs, sms, s) : launch_join_w<D, 1, 16>(p, pairs, sms, s);
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_tree_attention_workspace_bytes(const sv_kv_cache* cache, int B, const int32_t* row_offsets, int n_q_heads) {
  KvCache c;
  RowMap m;
  return ta_check_batch(cache, B, row_offsets, n_q_heads, &c, &m) ? 0 : ta_workspace_bytes(c);
}

int sv_tree_attention(const sv_kv_cache* cache, int B, const int32_t* row_offsets, const int32_t* kv_len,
                      const int32_t* block_table, int table_pages, const uint16_t* q, int ldq, int n_q_heads, float scale,
                      const uint64_t* tree_mask, uint16_t* out, int ldo, void* workspace, size_t workspace_bytes,
                      void* stream) {
  TreeAttnParams p;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  int st = ta_check_batch(cache, B, row_offsets, n_q_heads, &p.c, &p.map);
  if (!st) st = ta_check_call(&p, kv_len, block_table, table_pages, q, ldq, n_q_heads, scale, tree_mask, out, ldo);
  if (st) return st;
  const int sms = ta_sms();
  if (!workspace || !aligned(workspace, 256)) return fail(SV_EINVAL, "workspace must be non-null and 256-byte aligned");
  if (workspace_bytes < ta_workspace_bytes(p.c)) return fail(SV_EINVAL, "workspace too small: %zu < %zu", workspace_bytes, ta_workspace_bytes(p.c));
  if (!p.map.offs[B]) return SV_OK;
  p.partial = static_cast<float*>(workspace);
  p.stats = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ta_partial_bytes(sms, p.c.dim));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bool one_unit;
  st = ta_launch(&p, s, &one_unit);
  if (st || one_unit) return st;         // (an item of one unit is never dealt to two CTAs)
  const cudaError_t e = p.c.dim == 128 ? launch_join<128>(p, sms, s) : launch_join<64>(p, sms, s);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "tree attention launch");
}

}  // extern "C"
