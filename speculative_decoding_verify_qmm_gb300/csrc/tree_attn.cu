// Attention of the drafted rows over the paged cache.
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - max)
//
// One CTA per (row, query head): 128 tokens at a time, one per thread, their
// scores from the cache directly; a running maximum and sum; then the values,
// two threads per 64-bit pair of a head's elements.
#include <cmath>

#include "sv_kv.cuh"

namespace sv {

struct TreeAttnParams {
  KvCache c;
  RowMap map;
  const int32_t *kv_len, *table;
  int table_pages;
  const __nv_bfloat16* q; int ldq;
  int group;                 // query heads per key head
  float scale;
  const uint64_t* mask;
  __nv_bfloat16* out; int ldo;
};

template <int BITS>
__device__ __forceinline__ float kv_value(const uint8_t* codes, const __half* s, const __half* b, size_t tok, int dim, int d) {
  if constexpr (BITS == 16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(codes)[tok * dim + d]);
  const size_t g = tok * (dim / GROUP) + d / GROUP;
  const uint32_t code = BITS == 8 ? codes[tok * dim + d] : (codes[(tok * dim + d) >> 1] >> (4 * (d & 1))) & 15u;
  return fmaf(__half2float(s[g]), (float)code, __half2float(b[g]));
}

template <int BITS>
__global__ void __launch_bounds__(128) tree_attn_kernel(const __grid_constant__ TreeAttnParams p) {
  __shared__ float s_q[128], s_p[128], s_red[8];
  __shared__ size_t s_tok[128];
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, hq = blockIdx.y, h = hq / p.group, tid = threadIdx.x, D = p.c.dim;
  const int b = request_of(p.map, row), i = row - p.map.offs[b], m = p.map.offs[b + 1] - p.map.offs[b];
  long long len = p.kv_len[b];
  const long long cap = (long long)p.table_pages << p.c.page_shift;
  if (len < 0 || len + m > cap) {
    if (tid == 0) raise_error(ERR_BAD_INPUT);
    len = len < 0 ? 0 : cap - m;
    if (len < 0) return;
  }
  const uint64_t bits = p.mask ? p.mask[row] : (i == 63 ? ~0ull : (1ull << (i + 1)) - 1);
  if (tid < D) s_q[tid] = __bfloat162float(p.q[(size_t)row * p.ldq + hq * D + tid]);
  __syncthreads();
  float top = -INFINITY, sum = 0.f, acc = 0.f;
  for (long long t0 = 0; t0 < len + m; t0 += 128) {
    const long long t = t0 + tid;
    float sc = -INFINITY;
    const long long back = t - len;
    bool seen = t < len + m && (back < 0 || (bits >> back & 1));
    size_t tok = 0;
    if (t < len + m) {
      const long long page = kv_page_of(p.c, p.table, p.table_pages, b, t);
      if (page < 0) {
        raise_error(ERR_BAD_INPUT);
        seen = false;
      } else {
        tok = kv_token(p.c, (int)page, h, (int)(t & ((1ll << p.c.page_shift) - 1)));
      }
    }
    if (seen) {
      float a = 0.f;
      for (int d = 0; d < D; ++d) a += s_q[d] * kv_value<BITS>(p.c.p.k, p.c.p.ks, p.c.p.kb, tok, D, d);
      sc = a * p.scale;
    }
    float mx = sc;
    for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if ((tid & 31) == 0) s_red[tid >> 5] = mx;
    __syncthreads();
    const float now = fmaxf(top, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
    const float ref = now == -INFINITY ? 0.f : now;
    const float pt = seen ? expf(sc - ref) : 0.f;
    const float fix = top == -INFINITY ? 0.f : expf(top - ref);
    top = now;
    s_p[tid] = seen ? pt : -1.f;
    s_tok[tid] = tok;
    float ps = pt;
    for (int off = 16; off; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
    if ((tid & 31) == 0) s_red[4 + (tid >> 5)] = ps;
    __syncthreads();
    sum = sum * fix + (s_red[4] + s_red[5]) + (s_red[6] + s_red[7]);
    acc *= fix;
    if (tid < D)
      for (int u = 0; u < 128; ++u)
        if (s_p[u] != -1.f) acc += s_p[u] * kv_value<BITS>(p.c.p.v, p.c.p.vs, p.c.p.vb, s_tok[u], D, tid);
    __syncthreads();
  }
  if (tid < D) p.out[(size_t)row * p.ldo + hq * D + tid] = __float2bfloat16_rn(sum == 0.f ? 0.f : acc / sum);
}

static int check_heads(const KvCache& c, int n_q_heads) {
  if (c.dim != 64 && c.dim != 128) return fail(SV_EUNSUPPORTED, "attention needs head_dim 64 or 128 (got %d)", c.dim);
  if (n_q_heads < c.heads || n_q_heads % c.heads || n_q_heads / c.heads > 64)
    return fail(SV_EINVAL, "n_q_heads must be 1 to 64 times n_kv_heads (got %d, %d)", n_q_heads, c.heads);
  return SV_OK;
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_tree_attention_workspace_bytes(const sv_kv_cache* cache, int B, const int32_t* row_offsets, int n_q_heads) {
  KvCache c;
  RowMap m;
  if (check_cache(cache, &c) || check_rows_map(B, row_offsets, KV_MAX_DRAFT, 1 << 22, &m) || check_heads(c, n_q_heads)) return 0;
  return 256;
}

int sv_tree_attention(const sv_kv_cache* cache, int B, const int32_t* row_offsets, const int32_t* kv_len,
                      const int32_t* block_table, int table_pages, const uint16_t* q, int ldq, int n_q_heads, float scale,
                      const uint64_t* tree_mask, uint16_t* out, int ldo, void* workspace, size_t workspace_bytes,
                      void* stream) {
  TreeAttnParams p;
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
  const size_t need = sv_tree_attention_workspace_bytes(cache, B, row_offsets, n_q_heads);
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
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(p.map.offs[B], n_q_heads), dim3(128), 0, static_cast<cudaStream_t>(stream), attr);
  const cudaError_t e = p.c.bits == 16 ? cudaLaunchKernelEx(&cfg, tree_attn_kernel<16>, p)
                                       : (p.c.bits == 8 ? cudaLaunchKernelEx(&cfg, tree_attn_kernel<8>, p)
                                                        : cudaLaunchKernelEx(&cfg, tree_attn_kernel<4>, p));
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "tree attention launch");
}

}  // extern "C"
