// The paged KV cache: rows quantized as they are written, read back, and the
// accepted path of a draft tree moved to the front of the drafted region
// (mlx-dspark wiki page, "Architecture": the target keeps its KV state over
// rounds and rolls rejected drafts back; the pages give no layout, so the
// codes are in the weight format: affine, group 64, fp16 scale and bias).
//
// All three are bound by memory, or by launch latency for a drafted block.
// A thread owns 8 adjacent values of a head (16 bytes of bf16, 8 or 4 bytes of
// codes); a quantization group is 8 adjacent lanes, whose extremes meet by three
// shuffles, so a value is read once and never staged.
#include "sv_kv.cuh"

namespace sv {

constexpr float KV_FAR = 65280.f;  // bf16; with it scale * code + bias <= 65344 stays finite in fp16
constexpr int KV_THREADS = 256;

struct KvRows {
  KvCache c;
  RowMap map;
  const int32_t* first;     // position of each request's row 0
  const int32_t* table;
  int table_pages;
  uint16_t *k, *v;          // bf16 rows (read by append, written by read)
  int ldk, ldv;
  bool vec_k, vec_v;
};

__device__ __forceinline__ uint4 load8(const uint16_t* u, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(u);
  return make_uint4(u[0] | ((uint32_t)u[1] << 16), u[2] | ((uint32_t)u[3] << 16), u[4] | ((uint32_t)u[5] << 16),
                    u[6] | ((uint32_t)u[7] << 16));
}
__device__ __forceinline__ void store8(uint16_t* u, const uint4& x, bool vec) {
  if (vec) {
    *reinterpret_cast<uint4*>(u) = x;
    return;
  }
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    u[2 * e] = (uint16_t)w[e];
    u[2 * e + 1] = (uint16_t)(w[e] >> 16);
  }
}

// A thread's place: row, K or V, head, chunk of 8 values; false past the last row.
struct KvItem {
  int row, head, chunk, b;
  bool is_v, live;
  long long page;   // -1: bad input
  int place;
};
__device__ __forceinline__ KvItem kv_item(const KvRows& a) {
  const int chunks = a.c.dim / 8, per_row = 2 * a.c.heads * chunks;
  const long long idx = (long long)blockIdx.x * KV_THREADS + threadIdx.x;
  KvItem it;
  it.live = idx < (long long)a.map.offs[a.map.B] * per_row;
  it.row = it.live ? (int)(idx / per_row) : 0;
  const int r = it.live ? (int)(idx - (long long)it.row * per_row) : 0;
  it.is_v = r >= a.c.heads * chunks;
  const int hc = it.is_v ? r - a.c.heads * chunks : r;
  it.head = hc / chunks;
  it.chunk = hc - it.head * chunks;
  it.page = -1;
  it.place = 0;
  if (it.live) {
    it.b = request_of(a.map, it.row);
    const long long first = a.first[it.b];
    const long long pos = first + (it.row - a.map.offs[it.b]);
    if (first >= 0) it.page = kv_page_of(a.c, a.table, a.table_pages, it.b, pos);
    it.place = (int)(pos & ((1ll << a.c.page_shift) - 1));
    if (it.page < 0) raise_error(ERR_BAD_INPUT);
  }
  return it;
}

template <int BITS>
__global__ void __launch_bounds__(KV_THREADS) kv_append_kernel(const __grid_constant__ KvRows a) {
  pdl_trigger();
  pdl_wait();
  const KvItem it = kv_item(a);
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (it.live) {
    const uint16_t* src = it.is_v ? a.v + (size_t)it.row * a.ldv : a.k + (size_t)it.row * a.ldk;
    raw = load8(src + it.head * a.c.dim + it.chunk * 8, it.is_v ? a.vec_v : a.vec_k);
  }
  const bool ok = it.live && it.page >= 0;
  const size_t tok = ok ? kv_token(a.c, (int)it.page, it.head, it.place) : 0;
  if constexpr (BITS == 16) {
    if (ok) {
      uint8_t* base = it.is_v ? a.c.p.v : a.c.p.k;
      *reinterpret_cast<uint4*>(base + (tok * a.c.dim + it.chunk * 8) * 2) = raw;
    }
  } else {
    float x[8];
    const __nv_bfloat162* r2 = reinterpret_cast<const __nv_bfloat162*>(&raw);
    float lo = INFINITY, hi = -INFINITY;
    int nan = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f = e & 1 ? __bfloat162float(r2[e / 2].y) : __bfloat162float(r2[e / 2].x);
      nan |= f != f;
      x[e] = fminf(fmaxf(f, -KV_FAR), KV_FAR);
      lo = fminf(lo, x[e]);
      hi = fmaxf(hi, x[e]);
    }
#pragma unroll
    for (int off = 4; off; off >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
      nan |= __shfl_xor_sync(0xffffffffu, nan, off);
    }
    constexpr int TOP = (1 << BITS) - 1;
    // the format's own roundings, each IEEE: a host or torch program gets the same codes
    const __half s16 = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), (float)TOP));
    const __half b16 = __float2half_rn(lo);
    const float s = __half2float(s16), b = __half2float(b16);
    uint32_t w[2] = {0, 0};
    if (s > 0.f && !nan) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float c = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[e], b), s)), 0.f), (float)TOP);
        const uint32_t code = (uint32_t)c;
        if constexpr (BITS == 8) w[e / 4] |= code << (8 * (e % 4));
        else w[0] |= code << (4 * e);
      }
    }
    if (ok) {
      uint8_t* dst = (it.is_v ? a.c.p.v : a.c.p.k) + tok * (a.c.dim * BITS / 8) + it.chunk * BITS;
      if constexpr (BITS == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(dst) = w[0];
      if ((it.chunk & 7) == 0) {
        const size_t g = tok * (a.c.dim / GROUP) + it.chunk / 8;
        const __half q16 = __ushort_as_half((unsigned short)0x7fff);
        (it.is_v ? a.c.p.vs : a.c.p.ks)[g] = nan ? q16 : s16;
        (it.is_v ? a.c.p.vb : a.c.p.kb)[g] = nan ? q16 : b16;
      }
    }
  }
}

template <int BITS>
__global__ void __launch_bounds__(KV_THREADS) kv_read_kernel(const __grid_constant__ KvRows a) {
  pdl_trigger();
  pdl_wait();
  const KvItem it = kv_item(a);
  if (!it.live || it.page < 0) return;
  const size_t tok = kv_token(a.c, (int)it.page, it.head, it.place);
  const uint8_t* base = it.is_v ? a.c.p.v : a.c.p.k;
  uint4 out;
  if constexpr (BITS == 16) {
    out = *reinterpret_cast<const uint4*>(base + (tok * a.c.dim + it.chunk * 8) * 2);
  } else {
    const uint8_t* src = base + tok * (a.c.dim * BITS / 8) + it.chunk * BITS;
    uint32_t w[2] = {0, 0};
    if constexpr (BITS == 8) {
      const uint2 t = *reinterpret_cast<const uint2*>(src);
      w[0] = t.x;
      w[1] = t.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(src);
    }
    const size_t g = tok * (a.c.dim / GROUP) + it.chunk / 8;
    const float s = __half2float((it.is_v ? a.c.p.vs : a.c.p.ks)[g]);
    const float b = __half2float((it.is_v ? a.c.p.vb : a.c.p.kb)[g]);
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(&out);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t code = BITS == 8 ? (w[e / 4] >> (8 * (e % 4))) & 255u : (w[0] >> (4 * e)) & 15u;
      o[e] = __float2bfloat16_rn(fmaf(s, (float)code, b));
    }
  }
  uint16_t* dst = it.is_v ? a.v + (size_t)it.row * a.ldv : a.k + (size_t)it.row * a.ldk;
  store8(dst + it.head * a.c.dim + it.chunk * 8, out, it.is_v ? a.vec_v : a.vec_k);
}

// Commit.  Destination j never lies behind source j, and no destination j is the
// source of a later step i > j (path[i] > path[j] >= j), so a thread that owns a
// fixed slice of a token's bytes may read several sources ahead and still
// write in order; threads own disjoint slices and never meet.
constexpr int COMMIT_LAYERS = 64;   // caches per launch: their pointers ride in the launch parameters
constexpr int COMMIT_AHEAD = 8;

struct CommitParams {
  KvPtrs L[COMMIT_LAYERS];
  KvCache c;                        // sizes (pointers unused)
  const int32_t *kv_len, *table, *path, *path_len;
  int table_pages, max_path;
};

template <typename T>
__device__ __forceinline__ void move_slices(T* base, size_t stride_t, int lane_t, const long long* src, const long long* dst,
                                            int n, size_t head_off) {
  for (int j0 = 0; j0 < n; j0 += COMMIT_AHEAD) {
    T t[COMMIT_AHEAD];
#pragma unroll
    for (int i = 0; i < COMMIT_AHEAD; ++i)
      if (j0 + i < n) t[i] = base[(src[j0 + i] + head_off) * stride_t + lane_t];
#pragma unroll
    for (int i = 0; i < COMMIT_AHEAD; ++i)
      if (j0 + i < n) base[(dst[j0 + i] + head_off) * stride_t + lane_t] = t[i];
  }
}

__global__ void __launch_bounds__(KV_THREADS) kv_commit_kernel(const __grid_constant__ CommitParams p) {
  __shared__ long long s_src[KV_MAX_DRAFT], s_dst[KV_MAX_DRAFT];  // token index of head 0
  __shared__ int s_n, s_bad;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y, tid = threadIdx.x;
  if (tid == 0) s_n = s_bad = 0;
  __syncthreads();
  const int n = p.path_len[b];
  const long long len = p.kv_len[b];
  bool bad = n < 0 || n > p.max_path || (n > 0 && len < 0);
  if (!bad && tid < n) {
    const int at = p.path[(size_t)b * p.max_path + tid];
    const int before = tid ? p.path[(size_t)b * p.max_path + tid - 1] : -1;
    bad = at <= before || at < 0 || at >= KV_MAX_DRAFT;
    if (!bad) {
      const long long sp = kv_page_of(p.c, p.table, p.table_pages, b, len + at);
      const long long dp = kv_page_of(p.c, p.table, p.table_pages, b, len + tid);
      bad = sp < 0 || dp < 0;
      if (!bad && at != tid) {
        const long long mask = (1ll << p.c.page_shift) - 1;
        s_src[tid] = (long long)kv_token(p.c, (int)sp, 0, (int)((len + at) & mask));
        s_dst[tid] = (long long)kv_token(p.c, (int)dp, 0, (int)((len + tid) & mask));
        atomicAdd(&s_n, 1);
      }
    }
  }
  if (bad) s_bad = 1;
  __syncthreads();
  if (s_bad) {
    if (tid == 0) raise_error(ERR_BAD_INPUT);
    return;
  }
  const int moves = s_n;            // the last `moves` steps of the path: path[j] - j never shrinks along it
  if (!moves) return;
  const long long *src = s_src + (n - moves), *dst = s_dst + (n - moves);
  const KvPtrs L = p.L[blockIdx.z];
  const int row16 = p.c.dim * p.c.bits / 128;               // 16-byte slices of one head's token
  const int code_items = 2 * p.c.heads * row16;
  const int groups = p.c.dim / GROUP;
  const int items = code_items + (p.c.bits == 16 ? 0 : 4 * p.c.heads * groups);
  const int idx = blockIdx.x * KV_THREADS + tid;
  if (idx >= items) return;
  if (idx < code_items) {
    const int v = idx >= code_items / 2, r = v ? idx - code_items / 2 : idx;
    const int h = r / row16, c = r - h * row16;
    move_slices(reinterpret_cast<uint4*>(v ? L.v : L.k), (size_t)row16, c, src, dst, moves, (size_t)h << p.c.page_shift);
  } else {
    const int r = idx - code_items, per = p.c.heads * groups;
    const int a = r / per, h = (r - a * per) / groups, g = (r - a * per) - h * groups;
    __half* const arr[4] = {L.ks, L.kb, L.vs, L.vb};
    uint16_t* base = reinterpret_cast<uint16_t*>(a == 0 ? arr[0] : (a == 1 ? arr[1] : (a == 2 ? arr[2] : arr[3])));
    move_slices(base, (size_t)groups, g, src, dst, moves, (size_t)h << p.c.page_shift);
  }
}

// ------------------------------------------------------------------ host side
int check_cache(const sv_kv_cache* c, KvCache* out) {
  if (!c) return fail(SV_EINVAL, "cache must be non-null");
  if (c->bits != 4 && c->bits != 8 && c->bits != 16)
    return fail(SV_EUNSUPPORTED, "cache bits must be 4, 8 or 16 (got %d)", c->bits);
  if (c->head_dim < GROUP || c->head_dim > 256 || c->head_dim % GROUP)
    return fail(SV_EUNSUPPORTED, "cache head_dim must be a multiple of 64 up to 256 (got %d)", c->head_dim);
  if (c->page_size < 16 || c->page_size > 65536 || (c->page_size & (c->page_size - 1)))
    return fail(SV_EUNSUPPORTED, "page_size must be a power of two in [16, 65536] (got %d)", c->page_size);
  if (c->n_kv_heads < 1 || c->n_kv_heads > 256) return fail(SV_EINVAL, "n_kv_heads must be in [1, 256] (got %d)", c->n_kv_heads);
  if (c->n_pages < 1) return fail(SV_EINVAL, "n_pages must be >= 1 (got %d)", c->n_pages);
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(SV_EINVAL, "cache k and v must be non-null and 16-byte aligned");
  if (c->bits != 16) {
    const void* s[4] = {c->k_scales, c->k_biases, c->v_scales, c->v_biases};
    for (const void* p : s)
      if (!p || !aligned(p, 16)) return fail(SV_EINVAL, "cache scales and biases must be non-null and 16-byte aligned");
  }
  out->p.k = static_cast<uint8_t*>(c->k);
  out->p.v = static_cast<uint8_t*>(c->v);
  out->p.ks = reinterpret_cast<__half*>(c->k_scales);
  out->p.kb = reinterpret_cast<__half*>(c->k_biases);
  out->p.vs = reinterpret_cast<__half*>(c->v_scales);
  out->p.vb = reinterpret_cast<__half*>(c->v_biases);
  out->n_pages = c->n_pages;
  out->page_shift = 0;
  while ((1 << out->page_shift) < c->page_size) ++out->page_shift;
  out->heads = c->n_kv_heads;
  out->dim = c->head_dim;
  out->bits = c->bits;
  return SV_OK;
}

int check_rows_map(int B, const int32_t* row_offsets, int max_per_request, int max_total, RowMap* m) {
  if (B < 1 || B > MAX_BATCH) return fail(SV_EINVAL, "B must be in [1, 256] (got %d)", B);
  if (!row_offsets) return fail(SV_EINVAL, "row_offsets must be non-null");
  if (row_offsets[0] != 0) return fail(SV_EINVAL, "row_offsets[0] must be 0");
  for (int b = 0; b < B; ++b) {
    const long long n = (long long)row_offsets[b + 1] - row_offsets[b];
    if (n < 0) return fail(SV_EINVAL, "row_offsets must not decrease");
    if (n > max_per_request) return fail(SV_EUNSUPPORTED, "a request has %lld rows, more than %d", n, max_per_request);
  }
  if (row_offsets[B] > max_total) return fail(SV_EUNSUPPORTED, "%d rows, more than %d", row_offsets[B], max_total);
  m->B = B;
  for (int b = 0; b <= B; ++b) m->offs[b] = row_offsets[b];
  return SV_OK;
}

int check_table(const KvCache& c, const int32_t* lens, const int32_t* block_table, int table_pages) {
  if (!lens || !block_table || !aligned(lens, 4) || !aligned(block_table, 4))
    return fail(SV_EINVAL, "lengths and block_table must be non-null and aligned");
  if (table_pages < 1) return fail(SV_EINVAL, "table_pages must be >= 1 (got %d)", table_pages);
  if (((long long)table_pages << c.page_shift) > (1ll << 30))
    return fail(SV_EUNSUPPORTED, "table_pages * page_size must be <= 2^30");
  return SV_OK;
}

static int kv_rows_call(bool append, const sv_kv_cache* cache, int B, const int32_t* row_offsets, const int32_t* first,
                        const int32_t* table, int table_pages, uint16_t* k, int ldk, uint16_t* v, int ldv, void* stream) {
  KvRows a;
  int st = check_cache(cache, &a.c);
  if (!st) st = check_rows_map(B, row_offsets, 1 << 22, 1 << 22, &a.map);
  if (!st) st = check_table(a.c, first, table, table_pages);
  if (st) return st;
  if (!k || !v || !aligned(k, 2) || !aligned(v, 2)) return fail(SV_EINVAL, "k and v rows must be non-null and 2-byte aligned");
  if (ldk < a.c.heads * a.c.dim || ldv < a.c.heads * a.c.dim)
    return fail(SV_EINVAL, "ldk and ldv must be >= n_kv_heads * head_dim");
  if (!a.map.offs[B]) return SV_OK;
  a.first = first;
  a.table = table;
  a.table_pages = table_pages;
  a.k = k;
  a.v = v;
  a.ldk = ldk;
  a.ldv = ldv;
  a.vec_k = aligned(k, 16) && ldk % 8 == 0;
  a.vec_v = aligned(v, 16) && ldv % 8 == 0;
  const long long items = (long long)a.map.offs[B] * 2 * a.c.heads * (a.c.dim / 8);
  const long long blocks = (items + KV_THREADS - 1) / KV_THREADS;
  if (blocks > 0x7fffffffll) return fail(SV_EUNSUPPORTED, "too many values in one call");
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)blocks), dim3(KV_THREADS), 0, static_cast<cudaStream_t>(stream), attr);
  const int bits = a.c.bits;
  cudaError_t e;
  if (append)
    e = bits == 16 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<16>, a)
                   : (bits == 8 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<8>, a) : cudaLaunchKernelEx(&cfg, kv_append_kernel<4>, a));
  else
    e = bits == 16 ? cudaLaunchKernelEx(&cfg, kv_read_kernel<16>, a)
                   : (bits == 8 ? cudaLaunchKernelEx(&cfg, kv_read_kernel<8>, a) : cudaLaunchKernelEx(&cfg, kv_read_kernel<4>, a));
  return e == cudaSuccess ? SV_OK : cuda_fail(e, append ? "cache append launch" : "cache read launch");
}

}  // namespace sv

using namespace sv;

extern "C" {

int sv_kv_append(const sv_kv_cache* cache, int B, const int32_t* row_offsets, const int32_t* kv_len,
                 const int32_t* block_table, int table_pages, const uint16_t* k, int ldk, const uint16_t* v, int ldv,
                 void* stream) {
  return kv_rows_call(true, cache, B, row_offsets, kv_len, block_table, table_pages, const_cast<uint16_t*>(k), ldk,
                      const_cast<uint16_t*>(v), ldv, stream);
}

int sv_kv_read(const sv_kv_cache* cache, int B, const int32_t* row_offsets, const int32_t* first,
               const int32_t* block_table, int table_pages, uint16_t* k, int ldk, uint16_t* v, int ldv, void* stream) {
  return kv_rows_call(false, cache, B, row_offsets, first, block_table, table_pages, k, ldk, v, ldv, stream);
}

int sv_kv_commit(const sv_kv_cache* layers, int n_layers, int B, const int32_t* kv_len, const int32_t* block_table,
                 int table_pages, const int32_t* path, int max_path, const int32_t* path_len, void* stream) {
  if (!layers) return fail(SV_EINVAL, "layers must be non-null");
  if (n_layers < 1 || n_layers > 1024) return fail(SV_EINVAL, "n_layers must be in [1, 1024] (got %d)", n_layers);
  if (B < 1 || B > MAX_BATCH) return fail(SV_EINVAL, "B must be in [1, 256] (got %d)", B);
  if (max_path < 1 || max_path > KV_MAX_DRAFT) return fail(SV_EINVAL, "max_path must be in [1, 64] (got %d)", max_path);
  CommitParams p;
  KvCache c;
  for (int l = 0; l < n_layers; ++l) {  // every layer is checked before anything is launched
    const int st = check_cache(layers + l, l ? &c : &p.c);
    if (st) return st;
    if (l && (c.n_pages != p.c.n_pages || c.page_shift != p.c.page_shift || c.heads != p.c.heads || c.dim != p.c.dim ||
              c.bits != p.c.bits))
      return fail(SV_EINVAL, "layer %d's cache differs in size or bits from layer 0's", l);
  }
  const int st = check_table(p.c, kv_len, block_table, table_pages);
  if (st) return st;
  if (!path || !path_len || !aligned(path, 4) || !aligned(path_len, 4))
    return fail(SV_EINVAL, "path and path_len must be non-null and aligned");
  p.kv_len = kv_len;
  p.table = block_table;
  p.path = path;
  p.path_len = path_len;
  p.table_pages = table_pages;
  p.max_path = max_path;
  const int items = 2 * p.c.heads * (p.c.dim * p.c.bits / 128) + (p.c.bits == 16 ? 0 : 4 * p.c.heads * (p.c.dim / GROUP));
  for (int l0 = 0; l0 < n_layers; l0 += COMMIT_LAYERS) {
    const int n = n_layers - l0 < COMMIT_LAYERS ? n_layers - l0 : COMMIT_LAYERS;
    for (int l = 0; l < n; ++l) {
      check_cache(layers + l0 + l, &c);
      p.L[l] = c.p;
    }
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3((items + KV_THREADS - 1) / KV_THREADS, B, n), dim3(KV_THREADS), 0,
                                        static_cast<cudaStream_t>(stream), attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_commit_kernel, p);
    if (e != cudaSuccess) return cuda_fail(e, "cache commit launch");
  }
  return SV_OK;
}

}  // extern "C"
