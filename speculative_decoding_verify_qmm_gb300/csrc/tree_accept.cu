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
// Measured (vocabulary 151936, in a graph): one tree of 32 nodes with the head's statistics 24 us; 24 trees of up to 64 nodes from raw logits
// 88 to 112 by their uniforms, which say how far a walk goes (alone, the longest among them take 58: a node some 8 us, a rejection 4, of which
// an exchange between CTAs is 1 to 1.5); 8 trees of 24 nodes, truncated to 64 tokens, 45 to 52 (25 a node: E and bins 5, the bins' sum 3,
// candidates and their order 7, exchanges and the draw the rest); 4 greedy trees of 16 nodes 9.6.  Issue slots are a quarter full at most, and
// neither prefetching likely rows to the L2 cache nor more loads in flight helps: chains of 64-bit arithmetic, barriers and exchanges.
//
// Weights are 64-bit integers in units of 2^-40: their sums do not depend on any order, a draw compares integers, and the
// cumulative sums are exact to some 2^-40 of the largest weight, where sums of fp32 terms (2^-24) would choose another token than
// the formula for one draw in some hundreds over a flat distribution.
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <type_traits>

#include "sv_kv.cuh"
#include "sv_kernels.h"

namespace sv {

constexpr int TV_THREADS = 512;
// Vocabulary elements per thread whose loads are in flight together: where sums are made, and where a row is only read.  (24 trees of 64 nodes,
// one tree, four greedy ones, us: 7 and 20 105, 23.7, 9.4; 10 and 10 112, 24.1, 9.8; 13 and 20 106, 24.9, 9.4; 20 and 20 113, 24.7, 9.4.)
constexpr int TV_BATCH = 7;
constexpr int TV_READ = 20;
constexpr int TV_UNIT = 40;              // weights count in 2^-40 of the largest
constexpr int TV_MAX_V = 1 << 22;        // sums stay below 2^62
constexpr int TV_MAX_CLUSTER = 16;
constexpr int TV_BINS = 512;             // of a truncated row: bins of 1/16 in the exponent, 32 in all (e^-32 is below half a unit)
constexpr float TV_PER_E = 16.f;
constexpr int TV_LIST = 4096;            // a truncated row's candidates that are sorted
constexpr size_t TV_SMEM = 200 * 1024;   // dynamic shared memory: a slice's weights (and, truncating, bins and list)

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
  int top_k; float top_p;                // a truncated target (V and 1: not)
};

// 2^(i / 128) in two floats: square roots of 2, then products, in integers.
struct TvTable { float2 at[128]; };
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
  u64 root = 1ull << 63;                       // 2, in units of 2^-62
  for (int i = 0; i < 7; ++i) root = tv_sqrt((unsigned __int128)root << 62);
  unsigned __int128 x = (unsigned __int128)1 << 62;
  for (int i = 0; i < 128; ++i) {
    const double d = (double)(u64)x / (double)(1ull << 62);
    t.at[i].x = (float)d;
    t.at[i].y = (float)(d - (double)t.at[i].x);
    x = (x * root + ((unsigned __int128)1 << 61)) >> 62;
  }
  return t;
}
__constant__ TvTable g_tv_table = tv_table();

// x >> s, 0 for s > 63.
__device__ __forceinline__ u64 tv_shift(u64 x, int s) {
  u64 r;
  asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(x), "r"(s));
  return r;
}
// exp((z - top) / T) in units of 2^-40, off by 1.25 units at most (1.21 over 100 million values, rounded step by step on the host); 0 for
// -inf and NaN.  The exponent y = (z - top) log2(e) / T is held
// in two floats (the difference and the product exactly), y = N / 128 + r as in P. Tang's table-driven exponential (ACM TOMS 15, 1989):
// 2^(N/128) from the table, 2^r - 1 as g + g^2/2 + g^3/6 +
// g^4/24 of g = r ln 2, |g| < 2^-8.5, its first term and the result in two floats too.  Without branches: these would keep one element's
// chain from running beside another's.
__device__ __forceinline__ u64 tv_weight(float z, float top, float ch, float cl, const float2* table) {
  z = z > top ? top : z;                       // only if the caller's maximum is not one
  const float d = z - top, bb = d - z, lo = (z - (d - bb)) + (-top - bb);
  const float yh = d * ch, yl = fmaf(d, ch, -yh) + fmaf(d, cl, lo * ch);
  const float y = fmaxf(yh, -60.f);            // from -42 on nothing is left
  constexpr float MAGIC = 98304.f;             // 1.5 * 2^16: a float of its binade steps by 1 / 128
  const float t = y + MAGIC;
  const int N = (int)(__float_as_uint(t) & 0x7fffffu) - 0x400000;
  const float r = y - (t - MAGIC);
  const float gh = r * 0.693147182f, gl = fmaf(r, 0.693147182f, -gh) + fmaf(r, -1.90465421e-9f, yl * 0.693147182f);
  const float low = fmaf(gh * gh, fmaf(gh, fmaf(gh, 4.16666679e-2f, 0.166666672f), 0.5f), fmaf(gl, gh, gl));
  const float2 e = table[N & 127];
  const float p = e.x * gh, s = e.x + p;
  // (e.y gh is up to 2^-32.5: without it weights are off by up to 89 units)
  const float rest = ((e.x - s) + p) + (fmaf(e.x, gh, -p) + fmaf(e.x, low, fmaf(e.y, gh, e.y)));
  // s < 2 to 2^-24, the rest to 2^-41
  const u64 x = (u64)((long long)__float2int_rn(s * 0x1p24f) * 131072 + __float2int_rn(rest * 0x1p41f));
  return (tv_shift(x, -(N >> 7)) + 1) >> 1;
}

// A q in units of 2^-40, A = mant * 2^(exp - 63): rounded; far above every weight where it is large.
struct TvScale { u64 mant; int exp; };
__device__ __forceinline__ TvScale tv_scale(double a) {
  TvScale s = {0, 0};
  const u64 bits = (u64)__double_as_longlong(a);
  const int e = (int)(bits >> 52);             // (A is a sum of weights over 2^-40, never subnormal)
  if (e == 0 || e >= 0x800) return s;          // zero, or (after bad row sums) negative
  s.mant = ((bits & 0xfffffffffffffull) | 0x10000000000000ull) << 11;
  s.exp = e - 1023;
  return s;
}
__device__ __forceinline__ u64 tv_product(TvScale a, float q) {
  const uint32_t b = __float_as_uint(fmaxf(q, 0.f));                           // (a negative number or NaN counts as 0)
  const uint32_t m = (b << 8) | 0x80000000u;
  const u64 x = (a.mant >> 32) * m + (((a.mant & 0xffffffffull) * m) >> 32);   // mant * (24-bit mantissa) / 2^24
  // x * 2^(24 + exp - 63 + e - 150 + 40); of e = 0 nothing is left
  const int shift = 148 - a.exp - (int)(b >> 23);
  return (tv_shift(x, shift > 0 ? shift : 0) + 1) >> 1;
}
// floor(x f), and whether that is x f, of x below 2^62 and 0 <= f <= 1.
__device__ __forceinline__ u64 tv_times(u64 x, float f, bool* exact) {
  const uint32_t b = __float_as_uint(f), m = b < 0x800000u ? 0u : (b & 0x7fffffu) | 0x800000u;
  const u64 hi = __umul64hi(x, (u64)m << 40), lo = x * ((u64)m << 40);   // x m / 2^24
  const int shift = 126 - (int)(b >> 23);                               // f = m 2^(e - 150)
  const u64 r = shift < 0 ? x : tv_shift(hi, shift);                    // (below 0: 1)
  if (exact) *exact = shift < 0 || (lo == 0 && (shift > 63 ? hi == 0 : r << shift == hi));
  return r;
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
__device__ __forceinline__ u64 tv_warp_scan(u64 v) {   // inclusive
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, v, off);
    if ((int)(threadIdx.x & 31) >= off) v += o;
  }
  return v;
}
// e^(-x / 16) in units of 2^-40, to a few 2^-22.
__device__ __forceinline__ float tv_bin_weight(float x) { return exp2f(40.f - x * (1.44269504f / TV_PER_E)); }
__device__ __forceinline__ void st_peer_u64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
// Tokens in the order of a truncation, largest logit first, ties to the lower index: a larger place comes earlier.
__device__ __forceinline__ u64 tv_place(float z, int k) { return (u64)order_key(z) << 32 | (0xffffffffu - (uint32_t)k); }
__device__ __forceinline__ float tv_logit(u64 place) {
  const uint32_t key = (uint32_t)(place >> 32);
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

enum : int { TV_GREEDY, TV_SAMPLED, TV_CUT };      // a temperature of zero; the whole target; a truncated one
// What the walk asks of the CTAs next.
enum : int { TV_ENTER, TV_SUM, TV_DRAW, TV_DONE };

template <int MODE, bool CACHED>
__global__ void __launch_bounds__(TV_THREADS, 2) tree_accept_kernel(const __grid_constant__ TreeAcceptParams p) {
  constexpr int T = TV_THREADS, W = T / 32;
  constexpr bool TRUNC = MODE == TV_CUT, sampled = MODE != TV_GREEDY;
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __shared__ float2 s_table[128];
  __shared__ u64 s_parts[2][TV_MAX_CLUSTER], s_red[W], s_scan[W], s_kids[KV_MAX_DRAFT], s_tell[2];
  __shared__ int s_parent[KV_MAX_DRAFT], s_token[KV_MAX_DRAFT], s_arg[KV_MAX_DRAFT];
  __shared__ float s_u[KV_MAX_DRAFT], s_z[KV_MAX_DRAFT], s_q[KV_MAX_DRAFT], s_top[KV_MAX_DRAFT], s_sum[KV_MAX_DRAFT], s_e[KV_MAX_DRAFT];
  __shared__ int s_gone[KV_MAX_DRAFT], s_v, s_len, s_do, s_n_gone, s_drawn, s_last, s_listed;
  __shared__ double s_gone_at[KV_MAX_DRAFT], s_A;
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster_ctas(), rank = (int)cluster_rank(), b = blockIdx.x / C;
  const int r0 = p.offs[b], n = p.offs[b + 1] - r0, V = p.V;
  const int k0 = (int)((long long)rank * V / C), k1 = (int)((long long)(rank + 1) * V / C);
  const bool has_q = sampled && p.q != nullptr, stats = p.row_max != nullptr;
  // CACHED: E of the slice; truncating, before it the bins and the list of candidates
  unsigned* const s_bins = reinterpret_cast<unsigned*>(s_dyn);
  u64* const s_list = reinterpret_cast<u64*>(s_dyn + (TRUNC ? TV_BINS * 4 : 0));
  u64* const s_weight = s_list + (TRUNC ? TV_LIST : 0);
  if (tid < 128) s_table[tid] = g_tv_table.at[tid];
  cluster_sync();                                           // the others' shared memory is there from here on
  pdl_wait();
  // what the tests need of every node
  bool bad = false;
  if (tid < n) {
    const int up = tid ? p.parent[r0 + tid] : -1, x = tid ? p.token[r0 + tid] : 0;
    if (sampled) s_u[tid] = p.u[r0 + tid];
    if (stats && sampled) {
      s_top[tid] = p.row_max[r0 + tid];
      s_sum[tid] = p.row_sumexp[r0 + tid];
    } else if (stats) {
      s_arg[tid] = p.row_argmax[r0 + tid];
    }
    bad = tid && ((unsigned)up >= (unsigned)tid || (unsigned)x >= (unsigned)V);
    s_parent[tid] = up;
    s_token[tid] = x;
    if (has_q && tid && !bad) {
      const float z = p.logits[(size_t)(r0 + up) * p.ldl + x], top = stats ? p.row_max[r0 + up] : 0.f;
      s_q[tid] = p.q[(size_t)(r0 + up) * p.ldq + x];
      s_z[tid] = z;
      if (stats) s_e[tid] = expf((z - top) / p.temperature);
    }
  }
  if (__syncthreads_or(bad)) {                              // alike in all CTAs of the request
    if (rank == 0 && tid == 0) {
      raise_error(ERR_BAD_INPUT);
      p.out_len[b] = 0;
    }
    return;
  }
  for (int i = warp; i < n; i += W) {                       // each node's children
    const bool one = lane > 0 && lane < n && s_parent[lane] == i, two = 32 + lane < n && s_parent[(32 + lane) & 63] == i;
    const unsigned lo = __ballot_sync(0xffffffffu, one), hi = __ballot_sync(0xffffffffu, two);
    if (lane == 0) s_kids[i] = (u64)hi << 32 | lo;
  }
  __syncthreads();
  int turn = 0;                                             // exchanges so far: their buffer
  // The CTAs' values meet: every CTA has all of them afterwards.
  auto meet = [&](u64 mine, bool largest) -> const u64* {
    mine = largest ? tv_warp_max(mine) : tv_warp_sum(mine);
    if (lane == 0) s_red[warp] = mine;
    __syncthreads();
    u64* const parts = s_parts[turn++ & 1];
    if (warp == 0) {
      u64 x = lane < W ? s_red[lane] : 0;
      x = largest ? tv_warp_max(x) : tv_warp_sum(x);
      if (lane < C) st_peer_u64(peer(parts + rank, lane), x);
    }
    cluster_sync();
    return parts;
  };
  auto add = [&](const u64* parts) -> u64 {
    u64 all = 0;
    for (int c = 0; c < C; ++c) all += parts[c];
    return all;
  };

  // The walk, by thread 0 of every CTA: from the same numbers the same steps.  Everything else waits until it needs the others.
  int v = 0, len = 1, gone = 0;
  u64 rest = 0;                                             // children of v that have not been tried
  double A = 0.0, M = 0.0, left = 1.0;
  bool fresh = true, entered = false, told = false;         // at a new node; its M (or argmax) is known; its token is drawn
  // of the row at hand, alike in all threads
  int here = -1, arg = 0;                                   // node; its argmax
  float top = 0.f;
  u64 cut = 0, all = 0;                                     // TRUNC: the last place that is kept; the last sum
  bool near = false, have = false, summed = false;          // z, or E, is in shared memory; `all` and `parts` are those of A
  const u64* parts = nullptr;
  for (;;) {
    if (tid == 0) {
      auto follow = [&](int i) {                            // to child i, or the end
        if (rank == 0) {
          p.path[(size_t)b * p.max_path + len - 1] = v;
          p.out_tokens[r0 + len - 1] = s_token[i];
        }
        v = i;
        ++len;
        fresh = true;
      };
      auto match = [&](int token) -> int {
        for (u64 m = rest; m; m &= m - 1) {
          const int i = __ffsll((long long)m) - 1;
          if (s_token[i] == token) return i;
        }
        return -1;
      };
      int what = -1;
      while (what < 0) {
        if (fresh) {
          rest = len < p.max_path ? s_kids[v] : 0;
          A = 0.0;
          left = 1.0;
          gone = 0;
          fresh = told = false;
          entered = stats && !TRUNC;
          if (entered && has_q) M = (double)s_sum[v];
        }
        if (!has_q) {
          if (sampled ? !told : !entered) {
            what = sampled ? TV_DRAW : TV_ENTER;
            told = entered = true;
            break;
          }
          const int token = sampled ? s_drawn : (stats ? s_arg[v] : arg), i = match(token);
          if (i >= 0) {
            follow(i);
            continue;
          }
          what = TV_DONE;
          if (rank == 0) {
            p.path[(size_t)b * p.max_path + len - 1] = v;
            p.out_tokens[r0 + len - 1] = token;
            p.out_len[b] = len;
          }
          break;
        }
        if (!rest) {
          what = TV_DRAW;
          break;
        }
        if (!entered) {
          what = TV_ENTER;
          entered = true;
          break;
        }
        // A child after a rejected one needs the sum that is left; the sum before is not smaller, and a child that is accepted by that
        // needs no other.
        bool bound = false;
        const float Mf = (float)M;
        while (rest && !fresh && what < 0) {
          const int i = __ffsll((long long)rest) - 1, x = s_token[i];
          rest &= rest - 1;
          bool tried = false;
          for (int g = 0; g < gone; ++g) tried |= s_gone[g] == x;
          if (tried) continue;                              // without replacement a token comes once
          bool fits = false;
          if (!TRUNC || tv_place(s_z[i], x) >= cut) {
            // u q < W / M * left in fp32 (an exponent of up to 150 is off by 2^-16), in fp64 (slow here) where that does not tell
            const float leftf = (float)left, qx = s_q[i], taken = (float)A * qx, want = s_u[i] * qx * Mf, got = fmaxf(0.f, s_e[i] - taken) * leftf;
            const bool sure = fabsf(want - got) > 3e-5f * (want + (s_e[i] + taken) * leftf);
            fits = want < got && (sure || !bound);
            if (!sure && !bound) {
              const double e = exp(((double)s_z[i] - (double)(stats ? s_top[v] : top)) / (double)p.temperature);
              fits = (double)s_u[i] * (double)qx * M < fmax(0.0, e - A * (double)qx) * left;
            }
          }
          if (fits) {
            follow(i);
          } else if (bound) {
            rest |= 1ull << i;                              // to be tried with the sum
            what = TV_SUM;
          } else {
            if (p.distinct) {
              A += left == 1.0 ? M : M / left;
              left = fmax(left - (double)s_q[i], 0x1p-24);
              s_gone[gone] = x;
              s_gone_at[gone++] = A;
            } else {
              A += M;
            }
            bound = true;
          }
        }
        if (what < 0 && !fresh) what = bound ? TV_SUM : TV_DRAW;
      }
      s_v = v;
      s_len = len;
      s_do = what;
      s_A = A;
      s_n_gone = gone;
    }
    __syncthreads();
    const int what = s_do;
    if (what == TV_DONE) return;
    const int node = s_v, row = r0 + node;
    const float* const z = p.logits + (size_t)row * p.ldl;
    const float* const qr = has_q ? p.q + (size_t)row * p.ldq : nullptr;
    auto weight = [&](int k, float zk) -> u64 {
      if (TRUNC && cut && tv_place(zk, k) < cut) return 0;
      return tv_weight(zk, top, p.ch, p.cl, s_table);
    };
    // Sum of W = max(0, E - A q) over the vocabulary; each(k, z) sees the elements when E is made.
    auto total_of = [&](double D, int n_gone, auto each) {
      const TvScale a = tv_scale(D);
      u64 sum = 0;
      // what the loop does is fixed at compile time
      auto loop = [&](auto is_old, auto has_a) {
        constexpr bool OLD = decltype(is_old)::value, SUB = decltype(has_a)::value;
        auto batch = [&](int k, auto whole) {
          constexpr bool ALL = decltype(whole)::value;
          float x[OLD ? 1 : TV_BATCH], y[SUB ? TV_BATCH : 1];
#pragma unroll
          for (int i = 0; i < TV_BATCH; ++i) {
            const int kk = k + i * T;
            const bool in = ALL || kk < k1;
            if constexpr (!OLD) x[i] = !in ? 0.f : near ? *reinterpret_cast<const float*>(s_weight + (kk - k0)) : z[kk];
            if constexpr (SUB) y[i] = in ? qr[kk] : 0.f;
          }
#pragma unroll
          for (int i = 0; i < TV_BATCH; ++i) {
            const int kk = k + i * T;
            if (!OLD && !ALL && kk >= k1) continue;
            u64 w;
            if (OLD) {
              w = ALL || kk < k1 ? s_weight[kk - k0] : 0;   // (without branches)
            } else {
              w = weight(kk, x[i]);
              each(x[i]);
              if (CACHED) s_weight[kk - k0] = w;
            }
            if constexpr (SUB) w = tv_left(w, tv_product(a, y[i]));
            sum += w;
          }
        };
        int k = k0 + tid;
        for (; k + (TV_BATCH - 1) * T < k1; k += TV_BATCH * T) batch(k, std::true_type{});
        if (k < k1) batch(k, std::false_type{});
      };
      if (CACHED && have) {
        if (a.mant) loop(std::true_type{}, std::true_type{});
        else loop(std::true_type{}, std::false_type{});
      } else {
        if (a.mant) loop(std::false_type{}, std::true_type{});
        else loop(std::false_type{}, std::false_type{});
      }
      near = false;
      if (n_gone) {                                         // tokens that stay at the A of their own rejection
        __syncthreads();
        if (tid < n_gone && s_gone[tid] >= k0 && s_gone[tid] < k1) {
          const int k = s_gone[tid];
          const u64 w = CACHED ? s_weight[k - k0] : weight(k, z[k]);
          sum += tv_left(w, tv_product(tv_scale(s_gone_at[tid]), qr[k])) - tv_left(w, tv_product(a, qr[k]));
        }
      }
      have = true;
      parts = meet(sum, false);
      all = add(parts);
      summed = true;
    };
    auto total = [&](double D, int n_gone) { total_of(D, n_gone, [](float) {}); };

    if (node != here) {
      // ---------------------------------------------------------- a new row
      here = node;
      have = summed = false;
      cut = 0;
      top = stats && sampled ? s_top[node] : 0.f;
      if (!stats) {
        // its largest logit, lowest index first (its values stay in the weights' places)
        float best = -INFINITY;
        int at = k0 + tid < k1 ? k0 + tid : -1;
        for (int k = k0 + tid; k < k1; k += TV_READ * T) {
          float x[TV_READ];
#pragma unroll
          for (int i = 0; i < TV_READ; ++i) x[i] = k + i * T < k1 ? z[k + i * T] : -INFINITY;
#pragma unroll
          for (int i = 0; i < TV_READ; ++i) {
            const int kk = k + i * T;
            if (x[i] > best) {
              best = x[i];
              at = kk;
            }
            if (CACHED && kk < k1) *reinterpret_cast<float*>(s_weight + (kk - k0)) = x[i];
          }
        }
        near = CACHED;
        parts = meet(at < 0 ? 0 : tv_place(best, at), true);
        u64 most = 0;
        for (int c = 0; c < C; ++c) most = parts[c] > most ? parts[c] : most;
        top = tv_logit(most);
        arg = (int)(0xffffffffu - (uint32_t)most);
      }
      if constexpr (TRUNC) {
        // ---------------------------------------------------------- where the target is cut off
        for (int i = tid; i < TV_BINS; i += T) s_bins[i] = 0;
        if (tid == 0) s_listed = s_last = 0;
        __syncthreads();
        // natural exponents: the bins' limits are rounded, so what they decide leaves room for that
        const float scale = TV_PER_E * 0.693147182f * p.ch;
        total_of(0.0, 0, [&](float zk) {
          const float d = (top - zk) * scale;
          if (d < (float)TV_BINS) atomicAdd(s_bins + (d > 0.f ? (int)d : 0), 1u);
        });
        const u64 mass = all;
        // a bin a thread, the farthest first: tokens and mass (at most) behind it
        const int bin = TV_BINS - 1 - tid;
        unsigned count = 0;
        if (bin >= 0)
          for (int c0 = 0; c0 < C; c0 += 8) {
            unsigned x[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) x[c] = c0 + c < C ? ld_peer_u32(peer(s_bins + bin, c0 + c)) : 0u;
#pragma unroll
            for (int c = 0; c < 8; ++c) count += x[c];
          }
        const u64 mine = bin >= 0 ? (u64)((float)count * tv_bin_weight((float)bin)) : 0;
        const u64 tail_in = tv_warp_scan(mine), n_in = tv_warp_scan((u64)count);
        if (lane == 31) {
          s_red[warp] = tail_in;
          s_scan[warp] = n_in;
        }
        __syncthreads();
        u64 with = tail_in, farther = n_in - count, tokens = 0;
        for (int w = 0; w < W; ++w) {
          if (w < warp) {
            with += s_red[w];
            farther += s_scan[w];
          }
          tokens += s_scan[w];
        }
        // top_p: a bin is out if the mass from its near edge on is certainly less than what may be cut off
        const bool by_count = p.top_k < V;
        const bool in = by_count ? tokens - farther - count < (u64)p.top_k : !((double)with < (1.0 - (double)p.top_p) * (double)mass * 0.9375);
        if (in && count) atomicMax(&s_last, bin);
        __syncthreads();
        // the candidates: all tokens up to that bin's far edge, and a little more
        const u64 least = (u64)(tv_bin_weight((float)(s_last + 1)) * 0.998f);
        auto candidates = [&](auto take) {
#pragma unroll 4
          for (int k = k0 + tid; k < k1; k += T) {
            u64 w = CACHED ? s_weight[k - k0] : 0;
            if (CACHED && w < least) continue;
            const float zk = z[k];
            if (!CACHED) w = weight(k, zk);
            if (w >= least) take(tv_place(zk, k));
          }
        };
        int found = 0;
        candidates([&](u64) { ++found; });
        parts = meet((u64)found, false);
        int listed = 0, from = 0;
        for (int c = 0; c < C; ++c) {
          if (c < rank) from += (int)parts[c];
          listed += (int)parts[c];
        }
        if (listed == 0) {
          cut = 0;                                          // no token has weight
        } else if (listed <= TV_LIST) {
          candidates([&](u64 place) { st_peer_u64(peer(s_list + from + atomicAdd(&s_listed, 1), 0), place); });
          cluster_sync();
          if (rank == 0) {
            u64* sorted = s_list;
            if (listed <= T) {                              // each counts those before it
              sorted = s_list + T;
              const u64 mine = tid < listed ? s_list[tid] : 0;
              int before = 0;
              if (tid < listed) {
#pragma unroll 8
                for (int i = 0; i < listed; ++i) before += s_list[i] > mine;
                sorted[before] = mine;
              }
            } else {
              int size = T;
              while (size < listed) size <<= 1;
              for (int i = listed + tid; i < size; i += T) s_list[i] = 0;
              for (int k = 2; k <= size; k <<= 1)           // bitonic, largest place first
                for (int j = k >> 1; j; j >>= 1) {
                  __syncthreads();
                  for (int i = tid; i < size / 2; i += T) {
                    const int lo = ((i & ~(j - 1)) << 1) | (i & (j - 1)), hi = lo | j;
                    const u64 x = s_list[lo], y = s_list[hi];
                    if ((x < y) == !(lo & k)) {
                      s_list[lo] = y;
                      s_list[hi] = x;
                    }
                  }
                }
            }
            __syncthreads();
            // kept: rank below top_k, and mass before it below top_p of the first top_k's
            const int most = listed < p.top_k ? listed : p.top_k, per = (listed + T - 1) / T, i0 = tid * per;
            u64 sum = 0;
            for (int i = i0; i < i0 + per && i < most; ++i) sum += tv_weight(tv_logit(sorted[i]), top, p.ch, p.cl, s_table);
            const u64 inc = tv_warp_scan(sum);
            if (lane == 31) s_scan[warp] = inc;
            if (tid == 0) s_last = 0;
            __syncthreads();
            u64 before = inc - sum, firsts = 0;
            for (int w = 0; w < W; ++w) {
              if (w < warp) before += s_scan[w];
              firsts += s_scan[w];
            }
            bool exact;
            u64 limit = tv_times(by_count ? firsts : mass, p.top_p, &exact);
            limit += !exact;
            int kept = 0;
            for (int i = i0; i < i0 + per && i < most; ++i) {
              if (i > 0 && p.top_p < 1.f && before >= limit) break;
              before += tv_weight(tv_logit(sorted[i]), top, p.ch, p.cl, s_table);
              kept = i + 1;
            }
            if (kept) atomicMax(&s_last, kept);
            __syncthreads();
            if (tid < C) st_peer_u64(peer(s_tell, tid), sorted[s_last - 1]);
          }
          cluster_sync();
          cut = s_tell[0];
        } else {
          // Too many: the place is found bit by bit, by tokens, then by mass, with a pass over the row and an exchange for each of 64 bits.  Right
          // for any row, but slow.  (8 trees of 24 nodes, vocabulary 151936, logits of spread 2.5 at T = 0.75: top_p 0.8, which keeps some 1100,
          // 84 us in all; 0.9, where some rows have more than 4096 candidates, 491; 0.95 644, with a draft's distribution 1000 to 2300; top_k 20000 and
          // 0.95 959.)
          u64 lowest = 1;
          for (int by_mass = by_count ? 0 : 1; by_mass < (p.top_p < 1.f ? 2 : 1); ++by_mass) {
            const u64 floor_place = lowest;
            auto above = [&](u64 place) -> u64 {            // tokens from `place` on, or their mass
              u64 x = 0;
              for (int k = k0 + tid; k < k1; k += T) {
                const float zk = z[k];
                if (tv_place(zk, k) >= place) x += by_mass ? tv_weight(zk, top, p.ch, p.cl, s_table) : 1;
              }
              return add(meet(x, false));
            };
            const double want = by_mass ? (double)p.top_p * (double)(by_count ? above(floor_place) : mass) : (double)p.top_k;
            u64 place = 0;
            for (int bit = 63; bit >= 0; --bit) {
              const u64 t = place | 1ull << bit;
              if (t < floor_place || (double)above(t) >= want) place = t;
            }
            lowest = place > floor_place ? place : floor_place;
          }
          cut = lowest;
        }
        // what is cut off has no weight
        if (CACHED) {
#pragma unroll 4
          for (int k = k0 + tid; k < k1; k += T)
            if (s_weight[k - k0] < least || tv_place(z[k], k) < cut) s_weight[k - k0] = 0;
        }
        summed = false;
      }
    }
    if (what == TV_ENTER) {
      if (!sampled) continue;                               // (all that was wanted is the argmax)
      total(0.0, 0);
      if (!stats || TRUNC) {                                // the children's E, a lane each
        if (tid > 0 && tid < n && s_parent[tid] == node) {
          s_e[tid] = expf((s_z[tid] - top) / p.temperature);
        }
      }
      if (tid == 0) M = (double)all * (1.0 / (double)(1ull << TV_UNIT));
      __syncthreads();
      continue;
    }
    if (what == TV_SUM) {
      total(s_A, s_n_gone);
      if (all != 0) {
        if (tid == 0) M = (double)all * (1.0 / (double)(1ull << TV_UNIT));
        continue;
      }
    }
    // ------------------------------------------------------------ a draw
    double D = has_q ? s_A : 0.0;
    int n_gone = has_q ? s_n_gone : 0;
    if (summed && all == 0) {                               // no residual: from p
      D = 0.0;
      n_gone = 0;
      summed = false;
    }
    if (!summed) total(D, n_gone);
    const u64 base = tv_times(all, s_u[has_q ? 0 : node], nullptr);
    const u64 at = all == 0 ? 0 : (base < all ? base : all - 1);   // the first token whose cumulative sum is above
    u64 before = 0;
    int owner = 0;
    for (; owner < C - 1 && before + parts[owner] <= at; ++owner) before += parts[owner];
    int drawn = 0;
    if (rank == owner) {
      const TvScale a = tv_scale(D);
      // W of token k, where its own rejection counts
      auto remains = [&](int k, float zk, float qk) -> u64 {
        const u64 w = CACHED ? s_weight[k - k0] : weight(k, zk);
        for (int g = 0; g < n_gone; ++g)
          if (s_gone[g] == k) return tv_left(w, tv_product(tv_scale(s_gone_at[g]), qk));
        return tv_left(w, tv_product(a, qk));
      };
      if (CACHED && a.mant) {                               // in place, for the sums by ranges: this is the walk's end
        for (int k = k0 + tid; k < k1; k += TV_BATCH * T) {
          float y[TV_BATCH];
#pragma unroll
          for (int i = 0; i < TV_BATCH; ++i) y[i] = k + i * T < k1 ? qr[k + i * T] : 0.f;
#pragma unroll
          for (int i = 0; i < TV_BATCH; ++i)
            if (k + i * T < k1) s_weight[k + i * T - k0] = remains(k + i * T, 0.f, y[i]);
        }
        __syncthreads();
      }
      auto value = [&](int k) -> u64 {
        if (CACHED) return s_weight[k - k0];
        return a.mant ? remains(k, z[k], qr[k]) : weight(k, z[k]);
      };
      const int per = (k1 - k0 + T - 1) / T, a0 = min(k1, k0 + tid * per), a1 = min(k1, a0 + per);
      u64 mine = 0;
      for (int k = a0; k < a1; ++k) mine += value(k);
      const u64 inc = tv_warp_scan(mine);
      if (lane == 31) s_scan[warp] = inc;
      if (tid == 0) s_drawn = k1 > k0 ? k1 - 1 : V - 1;      // (no weight at all)
      __syncthreads();
      u64 run = before + inc - mine;
      for (int w = 0; w < warp; ++w) run += s_scan[w];
      if (run <= at && run + mine > at) {
        int k = a0;
        for (; k < a1 - 1; ++k) {
          run += value(k);
          if (run > at) break;
        }
        s_drawn = k;
      }
      __syncthreads();
      drawn = s_drawn;
    }
    if (has_q) {                                            // the end of the walk
      if (rank == owner && tid == 0) {
        p.out_tokens[r0 + s_len - 1] = drawn;
        p.out_len[b] = s_len;
        p.path[(size_t)b * p.max_path + s_len - 1] = node;
      }
      return;
    }
    if (rank == owner && tid < C) st_peer_u64(peer(s_tell + 1, tid), (u64)drawn);   // the owner tells the others
    cluster_sync();
    if (tid == 0) s_drawn = (int)s_tell[1];
  }
}

// ------------------------------------------------------------------ host side
template <int MODE, bool CACHED>
static cudaError_t launch_tree_accept_as(const TreeAcceptParams& p, int B, int C, size_t smem, cudaStream_t s) {
  const auto kernel = tree_accept_kernel<MODE, CACHED>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pdl_config(dim3(B * C), dim3(TV_THREADS), smem, s, attr);
  attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
  attr[cfg.numAttrs].val.clusterDim.x = C;
  attr[cfg.numAttrs].val.clusterDim.y = 1;
  attr[cfg.numAttrs].val.clusterDim.z = 1;
  ++cfg.numAttrs;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// The largest cluster that the device can place (16 is more than the portable 8).
static int tv_max_cluster() {
  static int cached = 0;
  if (cached) return cached;
  const auto kernel = tree_accept_kernel<TV_SAMPLED, true>;
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)TV_SMEM);
  cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  int c = TV_MAX_CLUSTER;
  for (; c > 8; c -= 4) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(TV_THREADS);
    cfg.dynamicSmemBytes = TV_SMEM;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0) break;
    cudaGetLastError();                  // clear a refusal; try a smaller cluster
  }
  return cached = c;
}

// CTAs a request: 16, for the shortest passes, while all requests are resident at once (two CTAs an SM), and 12 from there on, where fewer
// meetings count for more.  (A row of 151936; 16, 12, 8 and 4: 1 request 23.8 us, 26.7, 34.9 and 90; 9 requests 35, 44, 47 and 127; 16 from
// raw logits 90, 97, 106 and 193; 24 of 64 nodes 125, 127, 162 and 211, 64 of 16 nodes 225, 198, 257 and 267.)  The rule is made for large
// vocabularies.  (Of 32000: 1 request 16.5, 17.0, 19.8 and 26.8, 64 130, 97, 85 and 79; of 1000: 14.4, 13.9, 13.9 and 13.9, 64 106, 73, 52 and 36.)
static cudaError_t launch_tree_accept(const TreeAcceptParams& p, int B, cudaStream_t s) {
  const int most = tv_max_cluster(), C = B * 16 <= 2 * device_sm_count() || most < 12 ? most : 12;
  if (!(p.temperature > 0.f)) return launch_tree_accept_as<TV_GREEDY, false>(p, B, C, 0, s);
  const bool cut = p.top_k < p.V || p.top_p < 1.f;
  const size_t fixed = cut ? TV_BINS * 4 + TV_LIST * 8 : 0, slice = (size_t)((p.V + C - 1) / C) * 8;
  const bool cached = fixed + slice <= TV_SMEM;
  if (cut) return cached ? launch_tree_accept_as<TV_CUT, true>(p, B, C, fixed + slice, s) : launch_tree_accept_as<TV_CUT, false>(p, B, C, fixed, s);
  return cached ? launch_tree_accept_as<TV_SAMPLED, true>(p, B, C, slice, s) : launch_tree_accept_as<TV_SAMPLED, false>(p, B, C, 0, s);
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_tree_accept_workspace_bytes(int) { return 0; }

int sv_tree_accept(int B, const int32_t* row_offsets, const float* logits, int ldl, const float* row_max, const float* row_sumexp,
                   const int32_t* row_argmax, const int32_t* parent, const int32_t* token, const float* q, int ldq, int distinct, int V,
                   float temperature, const float* u, int top_k, float top_p, int32_t* out_len, int32_t* out_tokens, int32_t* path,
                   int max_path, void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace;                       // what a step keeps stays on the SMs
  (void)workspace_bytes;
  TreeAcceptParams p;
  memset(&p, 0, sizeof(p));
  RowMap map;
  int st = check_rows_map(B, row_offsets, KV_MAX_DRAFT, MAX_BATCH * KV_MAX_DRAFT, &map);
  if (st) return st;
  for (int b = 0; b < B; ++b)
    if (map.offs[b + 1] == map.offs[b]) return fail(SV_EINVAL, "request %d has no rows (the anchor is one)", b);
  if (V < 2 || V > TV_MAX_V) return fail(SV_EINVAL, "V must be in [2, 2^22] (got %d)", V);
  // (a difference of two logits that is beyond a float then has no weight)
  if (!(temperature >= 0.f && temperature <= 0x1p120f)) return fail(SV_EINVAL, "temperature must be in [0, 2^120]");
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
  // The CTAs of a request take the same steps because they read the same numbers; one of them writes while others may still read.
  const size_t rows = (size_t)map.offs[B];
  const struct { const void* at; size_t n; } arrays[] = {
      {out_len, (size_t)B}, {out_tokens, rows}, {path, (size_t)B * max_path},                     // what is written
      {parent, rows}, {token, rows}, {logits, (rows - 1) * ldl + V}, {row_max, rows}, {row_sumexp, rows}, {row_argmax, rows},
      {sampled ? u : nullptr, rows}, {sampled ? q : nullptr, (rows - 1) * ldq + V}};
  for (int i = 0; i < 3; ++i)
    for (const auto& x : arrays) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(arrays[i].at), c = reinterpret_cast<uintptr_t>(x.at);
      if (&x != &arrays[i] && x.at && a < c + 4 * x.n && c < a + 4 * arrays[i].n)
        return fail(SV_EINVAL, "out_len, out_tokens and path may not overlap each other or an input");
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
  p.top_k = top_k > 0 && top_k < V ? top_k : V;
  p.top_p = top_p;
  const cudaError_t e = launch_tree_accept(p, B, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "tree accept launch");
}

}  // extern "C"
