// Accept step of a draft tree (mlx-dspark releases page, v0.0.2 "Highlights", states the rule for a chain: accept with
// probability min(1, p / q), resample the residual; a tree tries a node's children in turn on what the ones before left).
//
// At a node with target p = exp((z - max) / T) / S and children drawn from q, in units where the largest p is 1:
//   W_1 = E = exp((z - max) / T),  M_1 = S,
//   child x is accepted iff u q_j(x) < W_j(x) / M_j, else W_j+1 = max(0, W_j - M_j q_j), M_j+1 = sum W_j+1,
// with q_j = q, or (children drawn without replacement) q without the tokens tried, divided by the mass left.  Since a
// subtraction after a clamp at 0 can be moved before it, W_j = max(0, E - A_j q) with A_1 = 0 and A_j+1 = A_j + M_j / mass left
// (a token tried without replacement stays at the A of its own rejection): a residual is one number, and a rejection one
// sum over the vocabulary.  Nothing is written back, and E is taken once per node.
//
// The walk down the tree is a chain of decisions, so the step is bound by latency: a cluster of CTAs shares a request, each
// with its slice of the vocabulary (E kept in shared memory), all of them take the same decisions from the same numbers, and
// meet only where a sum is needed.  What the tests need of every node is asked for at once before the walk begins.
//
// Weights are 64-bit integers in units of 2^-40: their sums do not depend on any order, a draw compares integers, and the
// cumulative sums are exact to some 2^-40 of the largest weight, where sums of fp32 terms (2^-24) would choose another token than
// the formula for one draw in some hundreds over a flat distribution.
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "sv_kv.cuh"
#include "sv_kernels.h"

namespace sv {

constexpr int TV_THREADS = 512, TV_WARPS = TV_THREADS / 32;
constexpr int TV_BATCH = 8;              // vocabulary elements per thread whose loads are in flight together
constexpr int TV_UNIT = 40;              // weights count in 2^-40 of the largest
constexpr int TV_CACHE = 24576;          // elements of a slice kept in shared memory
constexpr int TV_MAX_V = 1 << 22;        // sums stay below 2^62
constexpr int TV_MAX_CLUSTER = 16;

typedef unsigned long long u64;

struct TreeAcceptParams {
  int offs[MAX_BATCH + 1];
  const float* logits; int ldl;
  const float *row_max, *row_sumexp; const int32_t* row_argmax;
  const int32_t *parent, *token;
  const float* q; int ldq;
  int distinct, V;
  float temperature;
  float ch, cl;                          // log2(e) / T in two parts
  const float* u;
  int32_t *out_len, *out_tokens, *path; int max_path;
  const uint32_t* tkey; const int32_t* tidx; const float* tnorm;   // a truncated target's bounds (as in the chain's accept)
};

// 2^(i / 128) in units of 2^-62: square roots of 2, then products, in integers.
struct TvTable { u64 at[128]; };
constexpr u64 tv_sqrt(unsigned __int128 x) {   // floor, of x below 2^126
  u64 r = 0;
  for (int b = 62; b >= 0; --b) {
    const u64 t = r | (1ull << b);
    if ((unsigned __int128)t * t <= x) r = t;
  }
  return r;
}
constexpr TvTable tv_table() {
  TvTable t = {};
  u64 root = 1ull << 63;                       // 2
  for (int i = 0; i < 7; ++i) root = tv_sqrt((unsigned __int128)root << 62);
  unsigned __int128 x = (unsigned __int128)1 << 62;
  for (int i = 0; i < 128; ++i) {
    t.at[i] = (u64)x;
    x = (x * root + ((unsigned __int128)1 << 61)) >> 62;
  }
  return t;
}
__constant__ TvTable g_tv_table = tv_table();

// exp((z - top) / T) in units of 2^-40, off by one unit at most.  The exponent y = (z - top) log2(e) / T is held in two floats (the
// difference and the product exactly), y = N / 128 + r: 2^N/128 from the table, 2^r - 1 as g + g^2/2 + g^3/6 + g^4/24 of g = r ln 2,
// |g| < 2^-8.5, whose first term is in two floats too.
__device__ __forceinline__ u64 tv_weight(float z, float top, float ch, float cl, const u64* table) {
  if (z > top) z = top;                        // only if the caller's maximum is not one
  const float d = z - top, bb = d - z, lo = (z - (d - bb)) + (-top - bb);
  const float yh = d * ch;
  if (!(yh > -42.f)) return 0;                 // below a quarter of a unit (also -inf and NaN)
  const float yl = fmaf(d, ch, -yh) + fmaf(d, cl, lo * ch);
  constexpr float MAGIC = 98304.f;             // 1.5 * 2^16: a float of its binade steps by 1 / 128
  const float t = yh + MAGIC;
  const int N = (int)(__float_as_uint(t) & 0x7fffffu) - 0x400000;
  const float r = yh - (t - MAGIC);
  const float gh = r * 0.693147182f, gl = fmaf(r, 0.693147182f, -gh) + fmaf(r, -1.90465421e-9f, yl * 0.693147182f);
  const float low = fmaf(gh * gh, fmaf(gh, fmaf(gh, 4.16666679e-2f, 0.166666672f), 0.5f), fmaf(gl, gh, gl));
  const long long em = __float2ll_rn(gh * 2.81474977e14f) + __float2ll_rn(low * 2.81474977e14f);   // 2^48
  const u64 base = table[N & 127];
  const u64 x = base + (u64)__mul64hi((long long)base, em * 65536);
  const int shift = 62 - TV_UNIT - (N >> 7);
  return shift > 63 ? 0 : ((x >> (shift - 1)) + 1) >> 1;
}

// A q in units of 2^-40, A = mant * 2^(exp - 63): saturated, rounded.
struct TvScale { u64 mant; int exp; };
__device__ __forceinline__ TvScale tv_scale(double a) {
  TvScale s = {0, 0};
  if (!(a > 0.0)) return s;
  const u64 bits = (u64)__double_as_longlong(a);
  const int e = (int)(bits >> 52);
  s.mant = ((bits & 0xfffffffffffffull) | 0x10000000000000ull) << 11;   // (A is a sum of weights over 2^-40: normal)
  s.exp = e - 1023;
  return s;
}
__device__ __forceinline__ u64 tv_product(TvScale a, float q) {
  const uint32_t b = __float_as_uint(q);
  const int e = (int)(b >> 23);                // of a positive number; a negative one or NaN counts as 0 below
  if (a.mant == 0 || e == 0 || (int)b < 0 || q != q) return 0;
  const uint32_t m = (b << 8) | 0x80000000u;
  const u64 x = (a.mant >> 32) * m + (((a.mant & 0xffffffffull) * m) >> 32);   // mant * (24-bit mantissa) / 2^24
  const int shift = 149 - a.exp - e;           // x * 2^(24 + exp - 63 + e - 150 + 40)
  if (shift <= 0) return ~0ull >> 1;
  return shift > 63 ? 0 : ((x >> (shift - 1)) + 1) >> 1;
}
__device__ __forceinline__ u64 tv_left(u64 w, u64 taken) { return w > taken ? w - taken : 0; }

__device__ __forceinline__ u64 tv_warp_sum(u64 v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ u64 tv_warp_max(u64 v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    const u64 o = __shfl_xor_sync(0xffffffffu, v, off);
    v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ void st_peer_u64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

template <bool CACHED>
__global__ void __launch_bounds__(TV_THREADS) tree_accept_kernel(const __grid_constant__ TreeAcceptParams p) {
  extern __shared__ __align__(16) u64 s_weight[];          // CACHED: E of the slice
  __shared__ u64 s_table[128], s_parts[2][TV_MAX_CLUSTER], s_red[TV_WARPS], s_scan[TV_WARPS];
  __shared__ int s_parent[KV_MAX_DRAFT], s_token[KV_MAX_DRAFT], s_arg[KV_MAX_DRAFT];
  __shared__ float s_u[KV_MAX_DRAFT], s_z[KV_MAX_DRAFT], s_q[KV_MAX_DRAFT], s_top[KV_MAX_DRAFT], s_sum[KV_MAX_DRAFT];
  __shared__ int s_kid[KV_MAX_DRAFT], s_gone[KV_MAX_DRAFT], s_say[2];
  __shared__ double s_gone_at[KV_MAX_DRAFT], s_e[KV_MAX_DRAFT];
  __shared__ u64 s_draw[2];
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster_ctas(), rank = (int)cluster_rank(), b = blockIdx.x / C;
  const int r0 = p.offs[b], n = p.offs[b + 1] - r0, V = p.V;
  const int k0 = (int)((long long)rank * V / C), k1 = (int)((long long)(rank + 1) * V / C);
  const bool sampled = p.temperature > 0.f, has_q = sampled && p.q != nullptr, trunc = sampled && p.tkey != nullptr;
  const bool stats = p.row_max != nullptr;
  if (tid < 128) s_table[tid] = g_tv_table.at[tid];
  cluster_sync();                                           // the others' shared memory is there from here on
  pdl_wait();
  // what the tests need of every node
  bool bad = false;
  if (tid < n) {
    const int up = tid ? p.parent[r0 + tid] : -1, x = tid ? p.token[r0 + tid] : 0;
    bad = tid && ((unsigned)up >= (unsigned)tid || (unsigned)x >= (unsigned)V);
    s_parent[tid] = up;
    s_token[tid] = x;
    if (sampled) s_u[tid] = p.u[r0 + tid];
    if (stats) {
      if (sampled) {
        s_top[tid] = p.row_max[r0 + tid];
        s_sum[tid] = p.row_sumexp[r0 + tid];
      } else {
        s_arg[tid] = p.row_argmax[r0 + tid];
      }
    }
    if (trunc) s_sum[tid] = p.tnorm[r0 + tid];
    if (has_q && tid && !bad) {
      s_z[tid] = p.logits[(size_t)(r0 + up) * p.ldl + x];
      s_q[tid] = p.q[(size_t)(r0 + up) * p.ldq + x];
    }
  }
  if (__syncthreads_or(bad)) {                              // alike in all CTAs of the request
    if (rank == 0 && tid == 0) {
      raise_error(ERR_BAD_INPUT);
      p.out_len[b] = 0;
    }
    return;
  }
  int turn = 0;                                             // exchanges so far: their buffer
  // The CTAs' values meet: every CTA has all of them afterwards.
  auto meet = [&](u64 mine, bool largest) -> const u64* {
    mine = largest ? tv_warp_max(mine) : tv_warp_sum(mine);
    if (lane == 0) s_red[warp] = mine;
    __syncthreads();
    u64* const parts = s_parts[turn++ & 1];
    if (warp == 0) {
      u64 x = lane < TV_WARPS ? s_red[lane] : 0;
      x = largest ? tv_warp_max(x) : tv_warp_sum(x);
      if (lane < C) st_peer_u64(peer(parts + rank, lane), x);
    }
    cluster_sync();
    return parts;
  };

  int v = 0, len = 1;
  for (;;) {
    // ------------------------------------------------------------ a node
    const int row = r0 + v;
    const float* const z = p.logits + (size_t)row * p.ldl;
    const float* const qr = has_q ? p.q + (size_t)row * p.ldq : nullptr;
    // its children, in order
    if (warp == 0) {
      int count = 0;
#pragma unroll
      for (int h = 0; h < KV_MAX_DRAFT; h += 32) {
        const bool mine = h + lane < n && h + lane > 0 && s_parent[h + lane] == v;
        const unsigned m = __ballot_sync(0xffffffffu, mine);
        if (mine) s_kid[count + __popc(m & ((1u << lane) - 1))] = h + lane;
        count += __popc(m);
      }
      if (lane == 0) s_say[1] = len < p.max_path ? count : 0;
    }
    // the row's largest logit, lowest index first
    float top = stats && sampled ? s_top[v] : 0.f;
    int arg = stats && !sampled ? s_arg[v] : 0;
    if (!stats) {
      float best = -INFINITY;
      int at = k0 + tid < k1 ? k0 + tid : -1;
      for (int k = k0 + tid; k < k1; k += TV_BATCH * TV_THREADS) {
        float x[TV_BATCH];
#pragma unroll
        for (int i = 0; i < TV_BATCH; ++i) x[i] = k + i * TV_THREADS < k1 ? z[k + i * TV_THREADS] : -INFINITY;
#pragma unroll
        for (int i = 0; i < TV_BATCH; ++i)
          if (x[i] > best) {
            best = x[i];
            at = k + i * TV_THREADS;
          }
      }
      const u64* parts = meet(at < 0 ? 0 : (u64)order_key(best) << 32 | (0xffffffffu - (uint32_t)at), true);
      u64 most = 0;
      for (int c = 0; c < C; ++c) most = parts[c] > most ? parts[c] : most;
      const uint32_t key = (uint32_t)(most >> 32);
      top = __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
      arg = (int)(0xffffffffu - (uint32_t)most);
    }
    __syncthreads();
    const int kids = s_say[1];
    int next = -1, drawn = arg;
    if (sampled) {
      const uint32_t tK = trunc ? p.tkey[row] : 0u;
      const int tI = trunc ? p.tidx[row] : V;
      auto weight = [&](int k, float zk) -> u64 {
        if (trunc) {
          const uint32_t key = order_key(zk);
          if (!(key > tK || (key == tK && k <= tI))) return 0;
        }
        return tv_weight(zk, top, p.ch, p.cl, s_table);
      };
      bool have = false;                                    // E of this row is in shared memory
      double A = 0.0, left = 1.0;
      int gone = 0;
      // W of token k under the A of the moment, or of its own rejection
      auto remains = [&](int k) -> u64 {
        const u64 w = CACHED && have ? s_weight[k - k0] : weight(k, z[k]);
        if (!has_q) return w;
        double a = A;
        for (int g = 0; g < gone; ++g)
          if (s_gone[g] == k) a = s_gone_at[g];
        return a > 0.0 ? tv_left(w, tv_product(tv_scale(a), qr[k])) : w;
      };
      const u64* parts = nullptr;
      // sum of W over the vocabulary
      auto total = [&]() -> u64 {
        const TvScale a = tv_scale(A);
        u64 sum = 0;
        for (int k = k0 + tid; k < k1; k += TV_BATCH * TV_THREADS) {
          float x[TV_BATCH], y[TV_BATCH];
#pragma unroll
          for (int i = 0; i < TV_BATCH; ++i) {
            const int kk = k + i * TV_THREADS;
            x[i] = (!CACHED || !have) && kk < k1 ? z[kk] : 0.f;
            y[i] = a.mant && kk < k1 ? qr[kk] : 0.f;
          }
#pragma unroll
          for (int i = 0; i < TV_BATCH; ++i) {
            const int kk = k + i * TV_THREADS;
            if (kk >= k1) continue;
            u64 w;
            if (CACHED && have) {
              w = s_weight[kk - k0];
            } else {
              w = weight(kk, x[i]);
              if (CACHED) s_weight[kk - k0] = w;
            }
            sum += a.mant ? tv_left(w, tv_product(a, y[i])) : w;
          }
        }
        if (gone) {                                         // tokens that stay at the A of their own rejection
          __syncthreads();
          if (tid < gone && s_gone[tid] >= k0 && s_gone[tid] < k1) {
            const int k = s_gone[tid];
            const u64 w = CACHED ? s_weight[k - k0] : weight(k, z[k]);
            sum += tv_left(w, tv_product(tv_scale(s_gone_at[tid]), qr[k])) - tv_left(w, tv_product(a, qr[k]));
          }
        }
        have = true;
        parts = meet(sum, false);
        u64 all = 0;
        for (int c = 0; c < C; ++c) all += parts[c];
        return all;
      };
      constexpr double UNIT = 1.0 / (double)(1ull << TV_UNIT);
      bool summed = false;
      u64 all = 0;
      if (has_q) {
        double M;
        if (kids && (stats || trunc)) {
          M = (double)s_sum[v];
        } else {
          all = total();
          summed = true;
          M = (double)all * UNIT;
        }
        // the children's E, a lane each
        if (tid < kids) {
          const int i = s_kid[tid];
          const uint32_t key = order_key(s_z[i]);
          const bool kept = !trunc || key > tK || (key == tK && s_token[i] <= tI);
          s_e[tid] = kept ? exp(((double)s_z[i] - (double)top) / (double)p.temperature) : 0.0;
        }
        __syncthreads();
        for (int j = 0; j < kids && next < 0; ++j) {
          // every thread takes the decision, from the same numbers
          const int i = s_kid[j], x = s_token[i];
          bool tried = false;
          for (int g = 0; g < gone; ++g) tried |= s_gone[g] == x;
          if (tried) continue;                              // without replacement a token comes once
          const double qx = (double)s_q[i], w = fmax(0.0, s_e[j] - A * qx);
          if ((double)s_u[i] * qx * M < w * left) {
            next = i;
            break;
          }
          A += M / left;
          if (p.distinct) {
            left = fmax(left - qx, 0x1p-24);
            __syncthreads();                                // the list has been read
            if (tid == 0) {
              s_gone[gone] = x;
              s_gone_at[gone] = A;
            }
            ++gone;
            __syncthreads();
          }
          all = total();
          summed = true;
          M = (double)all * UNIT;
          if (all == 0) break;                              // nothing left to accept
        }
      }
      if (next < 0) {
        // ---------------------------------------------------------- a draw
        if (summed && all == 0) {                           // no residual: from p
          A = 0.0;
          gone = 0;
          summed = false;
        }
        if (!summed) all = total();
        const u64 base = (u64)((double)s_u[has_q ? 0 : v] * (double)all);
        const u64 at = all == 0 ? 0 : (base < all ? base : all - 1);   // the first token whose cumulative sum is above
        u64 before = 0;
        int owner = 0;
        for (; owner < C - 1 && before + parts[owner] <= at; ++owner) before += parts[owner];
        if (rank == owner) {
          const int per = (k1 - k0 + TV_THREADS - 1) / TV_THREADS, a0 = min(k1, k0 + tid * per), a1 = min(k1, a0 + per);
          u64 mine = 0;
          for (int k = a0; k < a1; ++k) mine += remains(k);
          u64 inc = mine;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const u64 o = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += o;
          }
          if (lane == 31) s_scan[warp] = inc;
          if (tid == 0) s_say[0] = k1 > k0 ? k1 - 1 : V - 1;  // (no weight at all)
          __syncthreads();
          u64 run = before + inc - mine;
          for (int w = 0; w < warp; ++w) run += s_scan[w];
          if (run <= at && run + mine > at) {
            int k = a0;
            for (; k < a1 - 1; ++k) {
              run += remains(k);
              if (run > at) break;
            }
            s_say[0] = k;
          }
          __syncthreads();
          drawn = s_say[0];
        }
        if (has_q) {                                        // the end of the walk
          if (rank == owner && tid == 0) {
            p.out_tokens[r0 + len - 1] = drawn;
            p.out_len[b] = len;
            p.path[(size_t)b * p.max_path + len - 1] = v;
          }
          return;
        }
        u64* const to = s_draw + (turn & 1);                // the owner tells the others
        if (rank == owner && tid < C) st_peer_u64(peer(to, tid), (u64)drawn);
        ++turn;
        cluster_sync();
        drawn = (int)*to;
      }
    }
    if (next < 0) {
      for (int j = kids - 1; j >= 0; --j)
        if (s_token[s_kid[j]] == drawn) next = s_kid[j];
    }
    if (rank == 0 && tid == 0) {
      p.path[(size_t)b * p.max_path + len - 1] = v;
      p.out_tokens[r0 + len - 1] = next < 0 ? drawn : s_token[next];
      if (next < 0) p.out_len[b] = len;
    }
    if (next < 0) return;
    v = next;
    ++len;
    __syncthreads();                                        // the node's lists have been read
  }
}

// ------------------------------------------------------------------ host side
template <bool CACHED>
static cudaError_t launch_tree_accept(const TreeAcceptParams& p, int B, int C, size_t smem, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(tree_accept_kernel<CACHED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && C > 8) e = cudaFuncSetAttribute(tree_accept_kernel<CACHED>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pdl_config(dim3(B * C), dim3(TV_THREADS), smem, s, attr);
  attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
  attr[cfg.numAttrs].val.clusterDim.x = C;
  attr[cfg.numAttrs].val.clusterDim.y = 1;
  attr[cfg.numAttrs].val.clusterDim.z = 1;
  ++cfg.numAttrs;
  return cudaLaunchKernelEx(&cfg, tree_accept_kernel<CACHED>, p);
}

static size_t tree_accept_bytes(int rows) { return align256((size_t)rows * 12); }

}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_tree_accept_workspace_bytes(int rows) { return rows < 1 || rows > MAX_BATCH * KV_MAX_DRAFT ? 0 : tree_accept_bytes(rows); }

int sv_tree_accept(int B, const int32_t* row_offsets, const float* logits, int ldl, const float* row_max, const float* row_sumexp,
                   const int32_t* row_argmax, const int32_t* parent, const int32_t* token, const float* q, int ldq, int distinct, int V,
                   float temperature, const float* u, int top_k, float top_p, int32_t* out_len, int32_t* out_tokens, int32_t* path,
                   int max_path, void* workspace, size_t workspace_bytes, void* stream) {
  TreeAcceptParams p;
  memset(&p, 0, sizeof(p));
  RowMap map;
  int st = check_rows_map(B, row_offsets, KV_MAX_DRAFT, MAX_BATCH * KV_MAX_DRAFT, &map);
  if (st) return st;
  for (int b = 0; b < B; ++b)
    if (map.offs[b + 1] == map.offs[b]) return fail(SV_EINVAL, "request %d has no rows (the anchor is one)", b);
  const int rows = map.offs[B];
  if (V < 2 || V > TV_MAX_V) return fail(SV_EINVAL, "V must be in [2, 2^22] (got %d)", V);
  if (!(temperature >= 0.f && temperature <= 3.4028235e38f)) return fail(SV_EINVAL, "temperature must be finite and >= 0");
  if (!logits || !parent || !token || !out_len || !out_tokens || !path) return fail(SV_EINVAL, "null pointer argument");
  for (const void* a : {(const void*)logits, (const void*)parent, (const void*)token, (const void*)q, (const void*)u, (const void*)row_max,
                        (const void*)row_sumexp, (const void*)row_argmax, (const void*)out_len, (const void*)out_tokens, (const void*)path})
    if (!aligned(a, 4)) return fail(SV_EINVAL, "arrays must be 4-byte aligned");
  if (ldl < V) return fail(SV_EINVAL, "ldl must be >= V");
  const bool sampled = temperature > 0.f;
  if (sampled && !u) return fail(SV_EINVAL, "a sampled accept needs u");
  if (sampled && q && ldq < V) return fail(SV_EINVAL, "ldq must be >= V");
  const int given = (row_max != nullptr) + (row_sumexp != nullptr) + (row_argmax != nullptr);
  if (given != 0 && given != 3 && !(!sampled && row_max && row_argmax))
    return fail(SV_EINVAL, "row statistics must be all given or all NULL");
  if (top_k < 0) return fail(SV_EINVAL, "top_k must be >= 0 (0 = no limit)");
  if (!(top_p > 0.f && top_p <= 1.f)) return fail(SV_EINVAL, "top_p must be in (0, 1]");
  if (max_path < 1 || max_path > KV_MAX_DRAFT) return fail(SV_EINVAL, "max_path must be in [1, 64] (got %d)", max_path);
  const bool trunc = sampled && ((top_k > 0 && top_k < V) || top_p < 1.f);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (trunc) {
    if (!workspace || !aligned(workspace, 256)) return fail(SV_EINVAL, "workspace must be non-null and 256-byte aligned");
    if (workspace_bytes < tree_accept_bytes(rows)) return fail(SV_EINVAL, "workspace too small: %zu < %zu", workspace_bytes, tree_accept_bytes(rows));
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    SelectArgs a;
    memset(&a, 0, sizeof(a));
    a.x = logits;
    a.ldx = ldl;
    a.V = V;
    a.mode = SEL_LOGITS;
    a.row_max = row_max;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.out_key = reinterpret_cast<uint32_t*>(ws);
    a.out_idx = reinterpret_cast<int32_t*>(ws + 4 * (size_t)rows);
    a.out_norm = reinterpret_cast<float*>(ws + 8 * (size_t)rows);
    const cudaError_t e = launch_select(a, rows, s);
    if (e != cudaSuccess) return cuda_fail(e, "truncation launch");
    p.tkey = a.out_key;
    p.tidx = a.out_idx;
    p.tnorm = a.out_norm;
  }
  for (int b = 0; b <= B; ++b) p.offs[b] = map.offs[b];
  p.logits = logits;
  p.ldl = ldl;
  p.row_max = row_max;
  p.row_sumexp = row_sumexp;
  p.row_argmax = row_argmax;
  p.parent = parent;
  p.token = token;
  p.q = q;
  p.ldq = ldq;
  p.distinct = distinct;
  p.V = V;
  p.temperature = temperature;
  if (sampled) {
    const double c = std::fmin(1.4426950408889634 / (double)temperature, 3.4028234663852886e38);
    p.ch = (float)c;
    p.cl = (float)(c - (double)p.ch);
  }
  p.u = u;
  p.out_len = out_len;
  p.out_tokens = out_tokens;
  p.path = path;
  p.max_path = max_path;
  const int C = 8;
  const int slice = (V + C - 1) / C;
  const cudaError_t e = slice <= TV_CACHE ? launch_tree_accept<true>(p, B, C, (size_t)slice * 8, s) : launch_tree_accept<false>(p, B, C, 0, s);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "tree accept launch");
}

}  // extern "C"
