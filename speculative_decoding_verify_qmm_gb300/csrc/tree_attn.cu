// Attention of the drafted rows over the paged cache: the entry point, and the join of items that spanned CTAs (the kernel
// itself is tree_attn_tc.cu).
#include <cmath>
#include <cstddef>
#include <cstring>

#include "tree_attn.cuh"

namespace sv {

constexpr int TA_MAX_BLOCK = 128, TA_NARROW_ROWS = 32;

// Joins the partial sums of items that spanned CTAs, in CTA order; a warp per (row, query head).
template <int D>
__global__ void __launch_bounds__(256) tree_attn_join_kernel(const __grid_constant__ TreeAttnParams p) {
  __shared__ TaPlan plan;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) ta_plan(p, &plan, false);
  __syncthreads();
  const int heads = p.c.heads * p.group;
  const long long id = (long long)blockIdx.x * 8 + warp;
  const int row = (int)(id / heads), hq = (int)(id - (long long)row * heads);
  if (row >= p.map.offs[p.map.B]) return;
  const int b = request_of(p.map, row), i = row - p.map.offs[b], m = p.map.offs[b + 1] - p.map.offs[b];
  const int h = hq / p.group, r = i * p.group + (hq - h * p.group), rb = r / p.block, k = r - rb * p.block;
  const int nt = (plan.len[b] + m + (1 << TA_UNIT_SHIFT) - 1) >> TA_UNIT_SHIFT;
  const long long units = plan.pre[p.map.B], per = (units + p.grid - 1) / p.grid;
  const long long a0 = plan.pre[b] + ((long long)h * ta_blocks(m * p.group, p.block) + rb) * nt;
  const int c0 = (int)(a0 / per), c1 = (int)((a0 + nt - 1) / per);
  if (c0 == c1) return;                                // one CTA had the whole item and wrote the output
  // CTA c's run of this item is its first one unless the item began inside the CTA's range
  auto slot_of = [&](int c) -> size_t { return 2 * (size_t)c + (c == c0 && a0 > (long long)c * per ? 1 : 0); };
  float most = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) most = fmaxf(most, p.stats[2 * slot_of(c) * p.block + k]);
#pragma unroll
  for (int off = 16; off; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
  const float base = most == -INFINITY ? 0.f : most;
  constexpr int E = D / 32;
  float acc[E] = {}, weight = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const size_t slot = slot_of(c);
    const float w = ta_exp2(p.stats[2 * slot * p.block + k] - base);
    weight += p.stats[(2 * slot + 1) * p.block + k] * w;
    const float* src = p.partial + (slot * p.block + k) * D + lane * E;
    float x[E];
    if constexpr (E == 4) {
      const float4 t = *reinterpret_cast<const float4*>(src);
      x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
    } else {
      const float2 t = *reinterpret_cast<const float2*>(src);
      x[0] = t.x; x[1] = t.y;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += x[e] * w;
  }
  __nv_bfloat16* dst = p.out + (size_t)row * p.ldo + hq * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(dst + e) =
        weight == 0.f ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(acc[e] / weight, acc[e + 1] / weight);
}

// ------------------------------------------------------------------ host side
static int check_heads(const KvCache& c, int n_q_heads) {
  if (c.dim != 64 && c.dim != 128) return fail(SV_EUNSUPPORTED, "attention needs head_dim 64 or 128 (got %d)", c.dim);
  if (n_q_heads < c.heads || n_q_heads % c.heads || n_q_heads / c.heads > 64)
    return fail(SV_EINVAL, "n_q_heads must be 1 to 64 times n_kv_heads (got %d, %d)", n_q_heads, c.heads);
  if ((long long)c.n_pages * c.heads > 0x7fffffffll) return fail(SV_EUNSUPPORTED, "n_pages * n_kv_heads must be below 2^31");
  return SV_OK;
}

// One CTA per SM (152 where no device is present: sizes only).
static int ta_sms() {
  const int n = device_sm_count();
  return n > 0 ? n : 152;
}
static size_t ta_partial_bytes(int grid, int dim) { return (size_t)2 * grid * TA_MAX_BLOCK * dim * sizeof(float); }
static size_t ta_stats_bytes(int grid) { return (size_t)4 * grid * TA_MAX_BLOCK * sizeof(float); }

template <int D>
static cudaError_t launch_join(const TreeAttnParams& p, cudaStream_t s) {
  const long long pairs = (long long)p.map.offs[p.map.B] * p.c.heads * p.group;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)((pairs + 7) / 8)), dim3(256), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, tree_attn_join_kernel<D>, p);
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_tree_attention_workspace_bytes(const sv_kv_cache* cache, int B, const int32_t* row_offsets, int n_q_heads) {
  KvCache c;
  RowMap m;
  if (check_cache(cache, &c) || check_rows_map(B, row_offsets, KV_MAX_DRAFT, 1 << 22, &m) || check_heads(c, n_q_heads)) return 0;
  return ta_partial_bytes(ta_sms(), c.dim) + ta_stats_bytes(ta_sms());
}

int sv_tree_attention(const sv_kv_cache* cache, int B, const int32_t* row_offsets, const int32_t* kv_len,
                      const int32_t* block_table, int table_pages, const uint16_t* q, int ldq, int n_q_heads, float scale,
                      const uint64_t* tree_mask, uint16_t* out, int ldo, void* workspace, size_t workspace_bytes,
                      void* stream) {
  TreeAttnParams p;
  memset(static_cast<void*>(&p), 0, offsetof(TreeAttnParams, c));
  int st = check_cache(cache, &p.c);
  if (!st) st = check_rows_map(B, row_offsets, KV_MAX_DRAFT, 1 << 22, &p.map);
  if (!st) st = check_table(p.c, kv_len, block_table, table_pages);
  if (!st) st = check_heads(p.c, n_q_heads);
  if (st) return st;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || ldq % 8 || ldo % 8)
    return fail(SV_EINVAL, "q and out must be non-null, 16-byte aligned, with strides that are multiples of 8");
  if (ldq < n_q_heads * p.c.dim || ldo < n_q_heads * p.c.dim) return fail(SV_EINVAL, "ldq and ldo must be >= n_q_heads * head_dim");
  if (!std::isfinite(scale)) return fail(SV_EINVAL, "scale must be finite");
  if (!aligned(tree_mask, 8)) return fail(SV_EINVAL, "tree_mask must be 8-byte aligned");
  const int sms = ta_sms();
  const size_t partial = ta_partial_bytes(sms, p.c.dim), need = partial + ta_stats_bytes(sms);
  if (!workspace || !aligned(workspace, 256)) return fail(SV_EINVAL, "workspace must be non-null and 256-byte aligned");
  if (workspace_bytes < need) return fail(SV_EINVAL, "workspace too small: %zu < %zu", workspace_bytes, need);
  if (!p.map.offs[B]) return SV_OK;
  p.kv_len = kv_len;
  p.table = block_table;
  p.table_pages = table_pages;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.ldq = ldq;
  p.group = n_q_heads / p.c.heads;
  p.scale = scale;
  p.mask = tree_mask;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.ldo = ldo;
  p.partial = static_cast<float*>(workspace);
  p.stats = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + partial);
  int rows = 0;                // of the widest request, times the group
  for (int b = 0; b < B; ++b) {
    const int m = p.map.offs[b + 1] - p.map.offs[b];
    if ((long long)m > ((long long)table_pages << p.c.page_shift))
      return fail(SV_EINVAL, "request %d has more rows than block_table has places", b);
    if (m * p.group > rows) rows = m * p.group;
  }
  // Items of up to 64 rows leave more shared memory to the ring of operand tiles; wider requests take items of 128.
  const bool narrow = rows <= TA_NARROW_ROWS;
  p.block = narrow ? (rows <= 16 ? 16 : 32) : (rows <= 64 ? 64 : TA_MAX_BLOCK);
  // the lengths are on the device: size the grid for the longest the table allows
  const long long most_units = (((long long)table_pages << p.c.page_shift) + (1 << TA_UNIT_SHIFT) - 1) >> TA_UNIT_SHIFT;
  long long most = 0;
  for (int b = 0; b < B; ++b)
    most += (long long)p.c.heads * ta_blocks((p.map.offs[b + 1] - p.map.offs[b]) * p.group, p.block) * most_units;
  p.grid = most < sms ? (int)most : sms;
  if (p.c.bits == 16 && !narrow) {
    const uint64_t slabs = (uint64_t)p.c.n_pages * p.c.heads, page = 1ull << p.c.page_shift;
    const uint32_t box = page < 128 ? (uint32_t)page : 128u;
    st = encode_tiled_3d_sw128(&p.tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.c.p.k, p.c.dim, page, slabs, 2, 64, box);
    if (!st) st = encode_tiled_3d_sw128(&p.tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.c.p.v, p.c.dim, page, slabs, 2, 64, box);
    if (st) return st;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = narrow ? launch_tree_attn_narrow(p, s) : launch_tree_attn(p, s);
  if (e == cudaSuccess && most_units > 1) e = p.c.dim == 128 ? launch_join<128>(p, s) : launch_join<64>(p, s);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "tree attention launch");
}

}  // extern "C"
