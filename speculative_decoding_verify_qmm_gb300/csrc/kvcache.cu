// The paged KV cache: rows quantized as they are written, read back, and the
// accepted path of a draft tree moved to the front of the drafted region
// (mlx-dspark wiki page, "Architecture": the target keeps its KV state over
// rounds and rolls rejected drafts back; the pages give no layout, so the
// codes are in the weight format: affine, group 64, fp16 scale and bias).
//
// All three are bound by memory, or by launch latency for a drafted block.
//
// Rows.  A thread owns 8 adjacent values of a head (16 bytes of bf16, 8 or 4
// bytes of codes), and the same ones of every row it works on, so that its heads,
// pointers and strides are set up once; a quantization group is 8 adjacent lanes.
// A value is read once and never staged.  A CTA takes tiles of consecutive rows; a
// row's request, page and place are looked up by one thread - the next tile's
// while the present one is worked on - and handed over in shared memory, for a
// lookup by every thread is three dependent loads against one load of data.
//
// Measured (8 heads of 128): 8253 rows written as 4-bit codes 14.8 us, as 8-bit codes 15.0, as bf16 12.8 (codes: 160
// instructions a warp for 8 values a lane are 9 us of issue, the rest waits, first for the barriers of a tile; bf16 by memory, 5.3 TB/s);
// read back 11.8 (100 instructions), 12.1 and 13.1; 32771 rows read from 8-bit codes 35.9 us (5.7 TB/s), from 4-bit codes 34.9, from
// bf16 44.6 (6.0 TB/s); 32 rows 2.2 us a call.  A lookup and two divisions by each thread, and a division a value, took 41 us to write
// and 74 for the long read.
#include "sv_kv.cuh"

#include <algorithm>
#include <functional>
#include <type_traits>

namespace sv {

constexpr float KV_FAR = 65280.f;  // bf16; with it scale * code + bias <= 65344 stays finite in fp16
constexpr int KV_THREADS = 256;    // at most
constexpr int KV_AHEAD = 4;        // chunks a thread has in flight when rows are many
// CTAs per SM of a long call: what is resident at once (read: 3 38.0 us, 4 36.1, 5 37.5, 6 49.0; append: 2 18.0, 3 15.9, 4 14.9).
constexpr int KV_APPEND_CTAS = 4;
constexpr int KV_READ_CTAS = 4;

struct KvRows {
  KvCache c;
  RowMap map;
  const int32_t* first;     // position of each request's row 0
  const int32_t* table;
  int table_pages;
  uint16_t *k, *v;          // bf16 rows (read by append, written by read)
  int ldk, ldv;
  bool vec_k, vec_v;
  int cols, step;           // chunks of a row (K's, then V's); rows that a CTA's threads cover at once
  int tile, tiles;          // rows of a tile
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

// Byte offset of a row's values in head 0; negative for bad input.
template <int BITS>
__device__ __forceinline__ long long kv_row_bytes(const KvRows& a, int row) {
  const int b = request_of(a.map, row);
  const int first = a.first[b];
  const long long pos = (long long)first + (row - a.map.offs[b]);
  const long long page = first < 0 ? -1 : kv_page_of(a.c, a.table, a.table_pages, b, pos);
  if (page < 0) {
    raise_error(ERR_BAD_INPUT);
    return -1;
  }
  return (long long)(kv_token(a.c, (int)page, 0, (int)(pos & ((1ll << a.c.page_shift) - 1))) * (a.c.dim * BITS / 8));
}

// What a thread owns of every row.
struct KvColumn {
  bool live, vec;
  int row, chunk;        // of the tile's rows, the first; chunk of the head
  uint8_t* data;         // its values in token 0
  __half *scale, *bias;
  uint16_t* rows;        // its values in row 0 of the caller's
  size_t ld;
};
template <int BITS>
__device__ __forceinline__ KvColumn kv_column(const KvRows& a) {
  KvColumn m;
  const int wide = min(a.cols, KV_THREADS);   // columns of a CTA
  m.row = threadIdx.x / wide;
  const int col = blockIdx.y * KV_THREADS + threadIdx.x - m.row * wide;
  m.live = m.row < a.step && col < a.cols;
  const int half = a.cols >> 1, chunks = a.c.dim / 8;
  const bool is_v = col >= half;
  const int hc = is_v ? col - half : col, head = hc / chunks;
  m.chunk = hc - head * chunks;
  const size_t tok = (size_t)head << a.c.page_shift;
  m.data = (is_v ? a.c.p.v : a.c.p.k) + tok * (a.c.dim * BITS / 8) + m.chunk * BITS;
  m.scale = (is_v ? a.c.p.vs : a.c.p.ks) + tok * (a.c.dim / GROUP) + m.chunk / 8;
  m.bias = (is_v ? a.c.p.vb : a.c.p.kb) + tok * (a.c.dim / GROUP) + m.chunk / 8;
  m.rows = (is_v ? a.v : a.k) + head * a.c.dim + m.chunk * 8;
  m.ld = is_v ? a.ldv : a.ldk;
  m.vec = is_v ? a.vec_v : a.vec_k;
  return m;
}
// A row's scales lie at 1 / (4 * BITS) of its codes' byte offset: 2 bytes for 64 codes.
template <int BITS>
__device__ __forceinline__ __half* kv_side(__half* base, long long bytes) {
  return reinterpret_cast<__half*>(reinterpret_cast<uint8_t*>(base) + (bytes >> (BITS == 8 ? 5 : 4)));
}

// The loop both kernels share.  work(rows, look) handles AHEAD rows at once: it calls look(offsets) for
// their byte offsets - after it has asked for the caller's rows, where it reads those - and ahead() once its
// loads are on their way: the CTA's next tile is looked up meanwhile.  All threads of a CTA make the same steps:
// work may shuffle.
template <int BITS, int AHEAD, typename Work>
__device__ __forceinline__ void kv_tiles(const KvRows& a, const KvColumn& m, Work work) {
  __shared__ long long s_at[2][KV_THREADS];
  const int tid = threadIdx.x, rows = a.map.offs[a.map.B];
  bool first = true;
  int buf = 0;
  for (int t = blockIdx.x; t < a.tiles; t += gridDim.x, buf ^= 1) {
    const int base = t * a.tile, n = min(a.tile, rows - base);
    for (int r0 = 0; r0 < a.tile; r0 += AHEAD * a.step) {
      int r[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) r[i] = r0 + m.row + i * a.step;
      work(base, r, n, [&](long long (&at)[AHEAD]) {
        if (first) {
          if (tid < n) s_at[0][tid] = kv_row_bytes<BITS>(a, base + tid);
          __syncthreads();
          first = false;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) at[i] = m.live && r[i] < n ? s_at[buf][r[i]] : -1;
      }, [&] {
        const int next = (t + (int)gridDim.x) * a.tile + tid;
        if (r0 == 0 && tid < a.tile && t + (int)gridDim.x < a.tiles && next < rows)
          s_at[buf ^ 1][tid] = kv_row_bytes<BITS>(a, next);
      });
    }
    __syncthreads();
  }
}

// bf16 number e of a chunk.
__device__ __forceinline__ float chunk_value(const uint4& r, int e) {
  const uint32_t u = e < 2 ? r.x : (e < 4 ? r.y : (e < 6 ? r.z : r.w));
  return __uint_as_float(e & 1 ? u & 0xffff0000u : u << 16);
}

template <int BITS, int AHEAD>
__global__ void __launch_bounds__(KV_THREADS, KV_APPEND_CTAS) kv_append_kernel(const __grid_constant__ KvRows a) {
  pdl_trigger();
  pdl_wait();
  const KvColumn m = kv_column<BITS>(a);
  const int lane = threadIdx.x & 31;
  kv_tiles<BITS, AHEAD>(a, m, [&](int base, const int (&r)[AHEAD], int n, auto look, auto ahead) {
    uint4 raw[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) raw[i] = make_uint4(0, 0, 0, 0);
    if (m.vec) {  // one branch, so that the loads leave together
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (m.live && r[i] < n) raw[i] = load8(m.rows + (size_t)(base + r[i]) * m.ld, true);
    } else {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (m.live && r[i] < n) raw[i] = load8(m.rows + (size_t)(base + r[i]) * m.ld, false);
    }
    long long at[AHEAD];
    look(at);
    ahead();
    if constexpr (BITS == 16) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (at[i] >= 0) *reinterpret_cast<uint4*>(m.data + at[i]) = raw[i];
    } else {
      constexpr int TOP = (1 << BITS) - 1;
      // Each group's extremes, as bf16 (exact) in pairs: (max, max of the negated).  A NaN stays.
      __nv_bfloat162 ends[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        auto pair = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
        const __nv_bfloat162 hi = __hmax2_nan(__hmax2_nan(pair(w[0]), pair(w[1])), __hmax2_nan(pair(w[2]), pair(w[3])));
        const __nv_bfloat162 lo = __hmin2_nan(__hmin2_nan(pair(w[0]), pair(w[1])), __hmin2_nan(pair(w[2]), pair(w[3])));
        ends[i] = __hmax2_nan(__halves2bfloat162(hi.x, __hneg(lo.x)), __halves2bfloat162(hi.y, __hneg(lo.y)));
      }
      // Over the 8 lanes of a group.  Of 4 groups a lane ends up with number lane % 4, so that the group's own
      // arithmetic is done once for the four: each exchange halves the groups a lane still reduces.
      auto other = [](__nv_bfloat162 x, int off) { return __hmax2_nan(x, __shfl_xor_sync(0xffffffffu, x, off)); };
      __nv_bfloat162 mine;
      if constexpr (AHEAD == 4) {
        const bool b0 = lane & 1, b1 = lane & 2;
        const __nv_bfloat162 s0 = __shfl_xor_sync(0xffffffffu, b0 ? ends[0] : ends[1], 1);
        const __nv_bfloat162 s1 = __shfl_xor_sync(0xffffffffu, b0 ? ends[2] : ends[3], 1);
        const __nv_bfloat162 p0 = __hmax2_nan(b0 ? ends[1] : ends[0], s0), p1 = __hmax2_nan(b0 ? ends[3] : ends[2], s1);
        const __nv_bfloat162 s2 = __shfl_xor_sync(0xffffffffu, b1 ? p0 : p1, 2);
        mine = other(__hmax2_nan(b1 ? p1 : p0, s2), 4);
      } else {
        static_assert(AHEAD == 1, "one group, or four");
        mine = other(other(other(ends[0], 1), 2), 4);
      }
      const float top = __bfloat162float(mine.x), bottom = -__bfloat162float(mine.y);
      const bool nan = top != top;
      const float hi = fminf(fmaxf(top, -KV_FAR), KV_FAR), lo = fminf(fmaxf(bottom, -KV_FAR), KV_FAR);
      // The format's own roundings, each IEEE: a host or torch program gets the same codes.
      const __half s16 = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), (float)TOP)), b16 = __float2half_rn(lo);
      const float s_mine = __half2float(s16);
      // A code is rint((x - b) / s) clamped to [0, TOP], the difference y and the quotient each rounded.  Ties
      // are common (bf16 values over an 11-bit scale), so the quotient must be the rounded one: by Markstein's
      // theorem (IBM J. Res. Dev. 34, 1990) t = y * inv, t + inv * (y - s * t) with two fused steps is that, for inv
      // = 1 / s rounded and s not all ones.  A group without a range, or with a NaN, has codes 0.
      const bool flat = !(s_mine > 0.f) || nan;
      const float inv_mine = flat ? 0.f : __fdiv_rn(1.f, s_mine);
      const uint32_t side_mine = nan ? 0x7fff7fffu : __half_as_ushort(s16) | ((uint32_t)__half_as_ushort(b16) << 16);
      // Without the clamp no code leaves [0, TOP] if every value is within KV_FAR and s is a normal number: s is off by
      // 2^-11 of itself, b by at most 2^-25.
      const bool odd = nan || top > KV_FAR || bottom < -KV_FAR || (s_mine > 0.f && s_mine < 6.103515625e-5f);
      const bool clamped = __any_sync(0xffffffffu, odd);
      constexpr float MAGIC = 12582912.f;  // 1.5 * 2^23: its sum with a small value rounds that to an integer, in the low bits
      uint32_t word[AHEAD][BITS / 4];
      auto codes = [&](auto clamp) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const float inv = AHEAD == 1 ? inv_mine : __shfl_sync(0xffffffffu, inv_mine, (lane & 24) + i);
          const uint32_t side = AHEAD == 1 ? side_mine : __shfl_sync(0xffffffffu, side_mine, (lane & 24) + i);
          const float s = inv > 0.f ? __half2float(__ushort_as_half((unsigned short)side)) : 0.f;
          const float b = __half2float(__ushort_as_half((unsigned short)(side >> 16)));
          uint32_t q[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float y = __fsub_rn(chunk_value(raw[i], e), b);
            // y instead of the code: both steps after it are monotonic.  s * TOP is exact (11 bits times 8)
            if constexpr (decltype(clamp)::value) y = fminf(fmaxf(y, 0.f), s * (float)TOP);
            const float t = __fmul_rn(y, inv);
            q[e] = __float_as_uint(__fadd_rn(fmaf(inv, fmaf(-s, t, y), t), MAGIC));
          }
          if constexpr (BITS == 8) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              word[i][e] = __byte_perm(__byte_perm(q[4 * e], q[4 * e + 1], 0x0040), __byte_perm(q[4 * e + 2], q[4 * e + 3], 0x0040), 0x5410);
          } else {  // the low 16 bits of each sum: MAGIC's own bits lie above them
            const uint32_t u = q[0] + 16u * q[1] + 256u * q[2] + 4096u * q[3], v = q[4] + 16u * q[5] + 256u * q[6] + 4096u * q[7];
            word[i][0] = __byte_perm(u, v, 0x5410);
          }
        }
      };
      if (clamped) codes(std::true_type{});
      else codes(std::false_type{});
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (at[i] < 0) continue;
        if constexpr (BITS == 8) *reinterpret_cast<uint2*>(m.data + at[i]) = make_uint2(word[i][0], word[i][1]);
        else *reinterpret_cast<uint32_t*>(m.data + at[i]) = word[i][0];
      }
      // each of a group's first AHEAD lanes has the scale and bias of one row
      const int own = lane & 7;
      long long mine_at = at[0];
      if constexpr (AHEAD == 4) mine_at = own & 2 ? (own & 1 ? at[3] : at[2]) : (own & 1 ? at[1] : at[0]);
      if (own < AHEAD && mine_at >= 0) {
        *kv_side<BITS>(m.scale, mine_at) = __ushort_as_half((unsigned short)side_mine);
        *kv_side<BITS>(m.bias, mine_at) = __ushort_as_half((unsigned short)(side_mine >> 16));
      }
    }
  });
}

template <int BITS, int AHEAD>
__global__ void __launch_bounds__(KV_THREADS, KV_READ_CTAS) kv_read_kernel(const __grid_constant__ KvRows a) {
  pdl_trigger();
  pdl_wait();
  const KvColumn m = kv_column<BITS>(a);
  kv_tiles<BITS, AHEAD>(a, m, [&](int base, const int (&r)[AHEAD], int, auto look, auto ahead) {
    long long at[AHEAD];
    look(at);
    uint4 raw[AHEAD];             // bf16, or codes in x (and y)
    __half scale[AHEAD], bias[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (at[i] < 0) continue;
      if constexpr (BITS == 16) {
        raw[i] = *reinterpret_cast<const uint4*>(m.data + at[i]);
      } else {
        if constexpr (BITS == 8) {
          const uint2 t = *reinterpret_cast<const uint2*>(m.data + at[i]);
          raw[i].x = t.x;
          raw[i].y = t.y;
        } else {
          raw[i].x = *reinterpret_cast<const uint32_t*>(m.data + at[i]);
        }
        scale[i] = *kv_side<BITS>(m.scale, at[i]);
        bias[i] = *kv_side<BITS>(m.bias, at[i]);
      }
    }
    ahead();
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if constexpr (BITS != 16) {
        const float s = __half2float(scale[i]), b = __half2float(bias[i]);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // a code in the low bits of 2^23 is that number plus 2^23
          uint32_t u;
          if constexpr (BITS == 8) u = __byte_perm(e < 4 ? raw[i].x : raw[i].y, 0x4b000000u, 0x7550 + e % 4);
          else u = ((raw[i].x >> (4 * e)) & 15u) | 0x4b000000u;
          x[e] = fmaf(s, __uint_as_float(u) - 8388608.f, b);
        }
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
          w[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (m.vec) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (at[i] >= 0) store8(m.rows + (size_t)(base + r[i]) * m.ld, raw[i], true);
    } else {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (at[i] >= 0) store8(m.rows + (size_t)(base + r[i]) * m.ld, raw[i], false);
    }
  });
}

// Commit.  Destination j never lies behind source j, and no destination j is the
// source of a later step i > j (path[i] > path[j] >= j), so a thread that owns a
// fixed slice of a token's bytes may read several sources ahead and still
// write in order; threads own disjoint slices and never meet.  Measured: 24 paths of 9 in 64 layers of 8 heads of 128, bf16,
// 12.7 us (5.0 TB/s); one path of 5 in 36 layers 2.5 us, a launch.
constexpr int COMMIT_LAYERS = 64;   // caches per launch: their pointers ride in the launch parameters
constexpr int COMMIT_AHEAD = 6;      // sources in flight per thread, and CTAs per SM: what 40 registers a thread allow
constexpr int COMMIT_CTAS = 6;       // (24 paths in 64 layers: 12.7 us; 8 and 5 12.8, 4 and 8 13.2, 8 and 6 15.7)

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

__global__ void __launch_bounds__(KV_THREADS, COMMIT_CTAS) kv_commit_kernel(const __grid_constant__ CommitParams p) {
  __shared__ long long s_src[KV_MAX_DRAFT], s_dst[KV_MAX_DRAFT];  // token index of head 0
  __shared__ int s_n, s_bad;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y, tid = threadIdx.x;
  // the path is asked for before its length is known: one wait less
  const int* path = p.path + (size_t)b * p.max_path;
  const int at = tid < p.max_path ? path[tid] : 0, before = tid && tid < p.max_path ? path[tid - 1] : -1;
  const int n = p.path_len[b];
  const long long len = p.kv_len[b];
  if (tid == 0) s_n = s_bad = 0;
  __syncthreads();
  bool bad = n < 0 || n > p.max_path || (n > 0 && len < 0);
  if (!bad && tid < n) {
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
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16) || c->k == c->v)
    return fail(SV_EINVAL, "cache k and v must be non-null, 16-byte aligned and not the same");
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
  const int sms = device_sm_count();
  if (sms <= 0) return fail(SV_ECUDA, "no CUDA device");
  const int rows = a.map.offs[B];
  a.cols = 2 * a.c.heads * (a.c.dim / 8);
  a.step = a.cols < KV_THREADS ? KV_THREADS / a.cols : 1;
  const int threads = a.cols < KV_THREADS ? (a.step * a.cols + 31) / 32 * 32 : KV_THREADS;
  const int wide = (a.cols + KV_THREADS - 1) / KV_THREADS;   // CTAs across a row
  // Few rows: a chunk per thread, for parallelism.  Many: KV_AHEAD of them at once, for bytes in flight.
  const bool many = (long long)rows * a.cols >= (long long)KV_AHEAD * KV_THREADS * sms;
  a.tile = a.step * (many ? KV_AHEAD : 1);
  const int most = (sms * (append ? KV_APPEND_CTAS : KV_READ_CTAS) + wide - 1) / wide;
  // A long read takes tiles of twice that, fewer lookups to wait for (32771 rows: 35.7 us against 36.6); where a CTA would have
  // less than two, they only balance worse (8253 rows written and read: 24.9 us against 26.2).
  if (many && !append && rows >= 4ll * a.tile * most) a.tile *= 2;
  a.tiles = (rows + a.tile - 1) / a.tile;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(a.tiles < most ? a.tiles : most, wide), dim3(threads), 0,
                                      static_cast<cudaStream_t>(stream), attr);
  using Kernel = void (*)(KvRows);
  static constexpr Kernel kernels[2][3][2] = {
      {{kv_read_kernel<4, 1>, kv_read_kernel<4, KV_AHEAD>},
       {kv_read_kernel<8, 1>, kv_read_kernel<8, KV_AHEAD>},
       {kv_read_kernel<16, 1>, kv_read_kernel<16, KV_AHEAD>}},
      {{kv_append_kernel<4, 1>, kv_append_kernel<4, KV_AHEAD>},
       {kv_append_kernel<8, 1>, kv_append_kernel<8, KV_AHEAD>},
       {kv_append_kernel<16, 1>, kv_append_kernel<16, KV_AHEAD>}}};
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernels[append][a.c.bits == 4 ? 0 : (a.c.bits == 8 ? 1 : 2)][many], a);
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
  // A cache listed twice would be moved twice at once.
  const void* seen[2 * 1024];
  for (int l = 0; l < n_layers; ++l) seen[2 * l] = layers[l].k, seen[2 * l + 1] = layers[l].v;
  std::sort(seen, seen + 2 * n_layers, std::less<const void*>());
  for (int i = 1; i < 2 * n_layers; ++i)
    if (seen[i] == seen[i - 1]) return fail(SV_EINVAL, "the same cache memory is listed twice");
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
