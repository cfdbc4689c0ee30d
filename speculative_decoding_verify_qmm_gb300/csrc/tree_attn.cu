// Attention of the drafted rows over the paged cache, on the 5th-generation
// tensor cores (mlx-dspark wiki page, "Architecture": the target verifies the
// drafted block in one forward over its cache).
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - max)
//
// The m drafted rows of a request times the query heads of one key head are up
// to 128 rows of one matrix (more: several row blocks); the cache is streamed
// past them in tiles of 128 tokens.  Bound by memory: a tile is D * bits / 4
// bytes per token against 4 * rows * D operations, and the tensor cores see the
// same 128-row instruction however few rows are real.
//
// Work: every (request, key head, row block) is an item of ceil(tokens / 128)
// tiles; the tiles of all items, in order, are dealt to one CTA per SM in equal
// contiguous runs, so ragged lengths balance and one long sequence fills the
// GPU.  An item that spans CTAs leaves fp32 partial sums (with their maximum and
// weight) in the workspace, and a second kernel joins them in CTA order.
//
// Per tile, S = Q K^T with Q (A operand) resident in tensor memory, K from
// shared memory, S [128 lanes x 128 tokens] in tensor memory; softmax of a lane
// by one thread; P (16 bits) back into tensor memory as the A operand of O += P V,
// V from shared memory as it lies ([token][dim], MN-major).  O stays in tensor
// memory; it is rescaled only when a row's maximum has grown by more than
// 2^6 since the last time, so the weights of the moment stay within 2^14.
//
// Few rows: with R <= 64 (32) rows the same rows are laid into 2 (4) groups of
// lanes, and each group takes its own half (quarter) of every tile's tokens - the
// off-diagonal blocks of P are zero - as an independent softmax that meets the
// others at the end of the item.  All four softmax warps then share the work
// that one would have had, without talking to each other.
//
// 16-bit caches go from TMA to the tensor cores untouched.  Codes are
// dequantized by eight warps into fp16 in the operand layout, fp16(s * c + b)
// with the exact code (half an fp16 step), and Q enters as fp16 scaled by a power
// of two per row, exact for every bf16 value within 2^29 of the row's largest.
#include <cmath>
#include <cstddef>
#include <cstring>

#include "sv_kv.cuh"
#include "sv_tc05.cuh"

namespace sv {

constexpr int TA_TILE = 128;                       // tokens per tile
constexpr int TA_ROWS = 128;                       // rows per block: the lanes of tensor memory
constexpr int TA_SOFT = 4, TA_XF = 8;              // softmax warps (0-3), transforming warps (4-11)
constexpr int TA_PROD = TA_SOFT + TA_XF, TA_MMA = TA_PROD + 1;
constexpr int TA_THREADS = (TA_MMA + 1) * 32;
constexpr int TA_PAD = 36;                         // floats per scratch row of 32 (16-byte aligned, conflict-free)
constexpr int TA_FLAGS = 16;                       // segments whose flags are alive at once (ring depth / 2 at most)
// tensor-memory columns
constexpr uint32_t TA_S = 0, TA_O = 256, TA_P = 384, TA_Q = 448;
constexpr float TA_BIAS = 8.f, TA_GROW = 14.f;     // weights start at 2^8 at most and may grow to 2^14

template <int D, int BITS>
struct TaShape {
  static constexpr int OP = TA_TILE * D * 2;                                       // one operand tile, 16 bits a value
  static constexpr int CODES = BITS == 16 ? 0 : TA_TILE * D * BITS / 8;            // one raw tile
  static constexpr int SIDE = BITS == 16 ? 0 : TA_TILE * (D / GROUP) * 2;          // its scales; its biases
  static constexpr int RAW = CODES + 2 * SIDE;
  static constexpr int SCRATCH = TA_ROWS * TA_PAD * 4;
  static constexpr int BUDGET = 222 * 1024 - SCRATCH - 1024;
  static constexpr int OPS = BITS == 16 ? (BUDGET / OP > 12 ? 12 : BUDGET / OP) : (D == 128 ? 3 : 4);
  static constexpr int RAWS_ALL = BITS == 16 ? 0 : (BUDGET - OPS * OP) / (RAW > 0 ? RAW : 1);
  static constexpr int RAWS = RAWS_ALL > 12 ? 12 : RAWS_ALL;
  static constexpr int SMEM = 1024 + OPS * OP + RAWS * RAW + SCRATCH;
  static constexpr int LOADS = BITS == 16 ? OPS : RAWS;                            // slots the copies land in
  static_assert(SMEM <= 224 * 1024, "shared memory");
  static_assert(LOADS <= 2 * TA_FLAGS - 4, "flags");
};

struct TreeAttnParams {
  CUtensorMap tk, tv;        // 16-bit caches: [pages * heads][page][dim], boxes of 64 x min(page, 128)
  KvCache c;
  RowMap map;
  const int32_t *kv_len, *table;
  int table_pages;
  const __nv_bfloat16* q; int ldq;
  int group;                 // query heads per key head
  float scale;
  const uint64_t* mask;
  __nv_bfloat16* out; int ldo;
  float* partial;            // [2 * grid][TA_ROWS][dim], then [2 * grid][2][TA_ROWS] (maximum, weight)
  float* stats;
  int grid;
};

// What every CTA of both kernels derives from the lengths: prefix sums of tiles.
struct TaPlan {
  long long pre[MAX_BATCH + 1];   // tiles of the requests before b
  int len[MAX_BATCH];             // committed tokens, brought into the table's range
};

__host__ __device__ __forceinline__ int ta_blocks(int m, int group) { return (m * group + TA_ROWS - 1) / TA_ROWS; }

// By one warp.
__device__ __forceinline__ void ta_plan(const KvCache& c, const RowMap& map, const int32_t* kv_len, int table_pages, int group,
                                        TaPlan* plan, bool report) {
  const int lane = threadIdx.x & 31;
  const long long cap = (long long)table_pages << c.page_shift;
  long long run = 0;
  for (int b0 = 0; b0 < map.B; b0 += 32) {
    const int b = b0 + lane;
    long long units = 0;
    if (b < map.B) {
      const int m = map.offs[b + 1] - map.offs[b];
      long long len = kv_len[b];
      if (m && (len < 0 || len + m > cap)) {
        if (report) raise_error(ERR_BAD_INPUT);
        len = len < 0 || cap < m ? 0 : cap - m;
      }
      plan->len[b] = (int)len;
      if (m) units = (long long)c.heads * ta_blocks(m, group) * ((len + m + TA_TILE - 1) / TA_TILE);
    }
    long long inc = units;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += up;
    }
    if (b < map.B) plan->pre[b + 1] = run + inc;
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) plan->pre[0] = 0;
}

// A run of tiles of one item in one CTA.
struct TaSeg {
  int b, h, rb, m, row0, rows;   // request, key head, row block; drafted rows, first row, rows of the block
  int tile0, n, nt, len, total;  // first tile, tiles, the item's tiles; committed and all tokens
  int split;                     // lane groups: 1, 2 or 4
  bool first;                    // starts at the CTA's first tile
};
__device__ __forceinline__ TaSeg ta_segment(const TreeAttnParams& p, const TaPlan& plan, long long u, long long u0, long long u1) {
  int lo = 0, hi = p.map.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (plan.pre[mid] <= u) lo = mid; else hi = mid;
  }
  TaSeg s;
  s.b = lo;                      // pre[lo] <= u < pre[lo + 1]: a request with tiles (the last of equal prefixes)
  s.row0 = p.map.offs[lo];
  s.m = p.map.offs[lo + 1] - s.row0;
  s.len = plan.len[lo];
  s.total = s.len + s.m;
  s.nt = (s.total + TA_TILE - 1) / TA_TILE;
  const unsigned long long local = (unsigned long long)(u - plan.pre[lo]);
  const int item = (int)(local / (unsigned)s.nt);
  s.tile0 = (int)(local - (unsigned long long)item * (unsigned)s.nt);
  const int nrb = ta_blocks(s.m, p.group);
  s.h = item / nrb;
  s.rb = item - s.h * nrb;
  const int left = s.m * p.group - s.rb * TA_ROWS;
  s.rows = left < TA_ROWS ? left : TA_ROWS;
  s.split = s.rows <= 32 ? 4 : (s.rows <= 64 ? 2 : 1);
  const long long can = u1 - u;
  s.n = s.nt - s.tile0 < can ? s.nt - s.tile0 : (int)can;
  s.first = u == u0;
  return s;
}

// Order of a segment's operand tiles: K0, K1, V0, K2, V1, ..., V(n-1).
__device__ __forceinline__ bool ta_item(int e, int n, int* tile) {
  if (e == 0) { *tile = 0; return false; }
  if (e == 2 * n - 1) { *tile = n - 1; return true; }
  if (e & 1) { *tile = (e + 1) / 2; return false; }
  *tile = e / 2 - 1;
  return true;
}

// Drafted tokens a row sees, as bits 0 .. m - 1.
__device__ __forceinline__ uint64_t ta_mask(const TreeAttnParams& p, int row, int i, int m) {
  const uint64_t all = m == 64 ? ~0ull : (1ull << m) - 1;
  return (p.mask ? p.mask[row] : (i == 63 ? ~0ull : (1ull << (i + 1)) - 1)) & all;
}

template <int BITS>
__device__ __forceinline__ float ta_cache_value(const uint8_t* codes, const __half* s, const __half* b, size_t tok, int dim, int d) {
  if constexpr (BITS == 16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(codes)[tok * dim + d]);
  const size_t g = tok * (dim / GROUP) + d / GROUP;
  const uint32_t code = BITS == 8 ? codes[tok * dim + d] : (codes[(tok * dim + d) >> 1] >> (4 * (d & 1))) & 15u;
  return fmaf(__half2float(s[g]), (float)code, __half2float(b[g]));
}

// One 32-bit word of codes as fp16 pairs s * c + b (two fp16 steps: an exact subtraction of 1024, one fused
// multiply-add).  8-bit: pairs (c0, c1), (c2, c3).  4-bit: pairs (c_j, c_j+4): inside each 8 elements position q holds
// element q / 2 + 4 (q % 2), an order that Q is laid out in too and that the output undoes.
template <int BITS>
__device__ __forceinline__ void ta_dequant(uint32_t w, __half2 s2, __half2 b2, uint32_t* out) {
  const __half2 k1024 = __half2half2(__ushort_as_half((unsigned short)0x6400));
#pragma unroll
  for (int j = 0; j < 16 / BITS; ++j) {
    const uint32_t biased = BITS == 8 ? __byte_perm(w, 0x64646464u, j ? 0x4342 : 0x4140)
                                      : (((w >> (4 * j)) & 0x000f000fu) | 0x64006400u);
    const __half2 v = __hfma2(s2, __hsub2(*reinterpret_cast<const __half2*>(&biased), k1024), b2);
    out[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
}
__device__ __forceinline__ bool ta_half_bad(uint32_t h) { return (h & 0x7c00u) == 0x7c00u; }

__device__ __forceinline__ float ta_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t ta_pack(float lo, float hi, bool bf16) {
  uint32_t r;
  if (bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A position in a ring of N slots and the parity of its current turn.
template <int N>
struct TaRing {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// A whole warp waits; false for all lanes once any gave up (the reason is recorded once).
__device__ __forceinline__ bool ta_wait(uint64_t* bar, uint32_t parity, volatile int* abort_v, unsigned err) {
  bool ok = mbar_wait_bounded(bar, parity, abort_v);
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) {
    if (!*abort_v) raise_error(err);
    *abort_v = 1;
  }
  return ok;
}

// Tiles whose V the transforming warps look through: those with drafted tokens or past the end.
__device__ __forceinline__ bool ta_fixed(const TaSeg& s, int j) { return (s.tile0 + j + 1) * TA_TILE > s.len; }

template <int D, int BITS>
__global__ void __launch_bounds__(TA_THREADS, 1) tree_attn_kernel(const __grid_constant__ TreeAttnParams p) {
  using Sh = TaShape<D, BITS>;
  constexpr bool RAW16 = BITS == 16;
  extern __shared__ uint8_t smem_raw[];
  // load_*: the slots that copies land in.  op_*: operand slots (the same ones for a 16-bit cache).
  __shared__ uint64_t load_full[12], load_empty[12], op_full[12], op_empty[12];
  __shared__ uint64_t q_full, s_full[2], p_full, pv_done, fin_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int abort_flag, s_bad[TA_FLAGS];
  __shared__ TaPlan plan;
  __shared__ float s_max[TA_ROWS], s_sum[TA_ROWS];
  __shared__ int s_ok[TA_SOFT];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const ops = smem;
  uint8_t* const raws = smem + Sh::OPS * Sh::OP;
  float* const scratch = reinterpret_cast<float*>(raws + Sh::RAWS * Sh::RAW);
  volatile int* abort_v = &abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::LOADS; ++i) {
      mbar_init(&load_full[i], 1);
      mbar_init(&load_empty[i], TA_XF);
    }
    for (int i = 0; i < Sh::OPS; ++i) {
      mbar_init(&op_full[i], TA_XF);
      mbar_init(&op_empty[i], 1);
    }
    mbar_init(&q_full, TA_SOFT);
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(&p_full, TA_SOFT);
    mbar_init(&pv_done, 1);
    mbar_init(&fin_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < TA_FLAGS) s_bad[threadIdx.x] = 0;
  if (warp == TA_MMA) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  pdl_wait();
  if (warp == 0) ta_plan(p.c, p.map, p.kv_len, p.table_pages, p.group, &plan, blockIdx.x == 0);
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  const uint32_t tmem = s_tmem;
  const long long units = plan.pre[p.map.B], per = (units + p.grid - 1) / p.grid;
  const long long u0 = blockIdx.x * per, u1 = u0 + per < units ? u0 + per : units;

  if (warp == TA_PROD) {
    // ============================================================ copies into the ring
    const int shift = p.c.page_shift < 7 ? p.c.page_shift : 7, chunk = 1 << shift;   // tokens per copy
    const int place_mask = (1 << p.c.page_shift) - 1;
    constexpr int PER = RAW16 ? D / 64 : 3;            // copies per chunk: 64-wide halves, or codes / scales / biases
    const int my_chunk = lane / PER, part = lane - my_chunk * PER;
    TaRing<Sh::LOADS> ring;
    bool ok = true;
    for (long long u = u0; u < u1 && ok;) {
      const TaSeg s = ta_segment(p, plan, u, u0, u1);
      // the page of this lane's chunk of tile j
      auto page_of = [&](int j) -> int {
        const int t = (s.tile0 + j) * TA_TILE + (my_chunk << shift);
        if (j >= s.n || my_chunk >= (TA_TILE >> shift) || t >= s.total) return 0;
        int page = p.table[(size_t)s.b * p.table_pages + (t >> p.c.page_shift)];
        if (page < 0 || page >= p.c.n_pages) {
          raise_error(ERR_BAD_INPUT);
          page = 0;                                    // stay inside the arrays: the result is undefined
        }
        return page;
      };
      // pages of the last two K tiles, and the next one's, fetched a tile ahead
      int page_before = 0, page_k = 0, page_next = page_of(0);
      for (int i = 0; i < 2 * s.n; ++i) {
        int j;
        const bool is_v = ta_item(i, s.n, &j);
        if (!is_v) {
          page_before = page_k;
          page_k = page_next;
          page_next = page_of(j + 1);
        }
        const int page = is_v && i != 2 * s.n - 1 ? page_before : page_k;
        ok = ta_wait(RAW16 ? &op_empty[ring.slot] : &load_empty[ring.slot], ring.phase ^ 1, abort_v, ERR_TIMEOUT_EMPTY);
        if (!ok) break;
        const int t0 = (s.tile0 + j) * TA_TILE;
        const int toks = s.total - t0 < TA_TILE ? s.total - t0 : TA_TILE;
        const int chunks = (toks + chunk - 1) >> shift;
        const uint32_t tx = (uint32_t)(chunks << shift) * (RAW16 ? D * 2 : D * BITS / 8 + 2 * (D / GROUP) * 2);
        if (lane == 0) mbar_arrive_expect_tx(&load_full[ring.slot], tx);
        __syncwarp();
        if (my_chunk < chunks) {
          const int place = (t0 + (my_chunk << shift)) & place_mask;
          if constexpr (RAW16) {
            uint8_t* dst = ops + ring.slot * Sh::OP + part * (TA_TILE * 128) + (my_chunk << shift) * 128;
            tma_load_3d_plain(dst, is_v ? &p.tv : &p.tk, &load_full[ring.slot], part * 64, place, page * p.c.heads + s.h);
          } else {
            const size_t tok = kv_token(p.c, page, s.h, place);
            uint8_t* raw = raws + ring.slot * Sh::RAW;
            if (part == 0) {
              const uint8_t* src = (is_v ? p.c.p.v : p.c.p.k) + tok * (D * BITS / 8);
              bulk_load_plain(raw + (my_chunk << shift) * (D * BITS / 8), src, (uint32_t)chunk * (D * BITS / 8),
                              &load_full[ring.slot]);
            } else {
              const __half* src = part == 1 ? (is_v ? p.c.p.vs : p.c.p.ks) : (is_v ? p.c.p.vb : p.c.p.kb);
              bulk_load_plain(raw + Sh::CODES + (part - 1) * Sh::SIDE + (my_chunk << shift) * (D / GROUP) * 2,
                              src + tok * (D / GROUP), (uint32_t)chunk * (D / GROUP) * 2, &load_full[ring.slot]);
            }
          }
        }
        ring.next();
      }
      u += s.n;
    }
    // every copy is waited for by its reader; after a failure, give those in flight time to land
    if (!ok || *abort_v) {
      const unsigned long long w0 = global_ns();
      while (global_ns() - w0 < 50000ull) __nanosleep(1000);
    }
  } else if (warp == TA_MMA) {
    // ============================================================ MMA issue
    if (lane == 0) {
      TaRing<Sh::OPS> ring;
      uint32_t n_q = 0, n_s = 0, n_p = 0;               // phases seen of each barrier
      bool ok = true;
      constexpr uint32_t ID_S = f16_idesc_ex(TA_ROWS, TA_TILE, RAW16, false);
      constexpr uint32_t ID_O = f16_idesc_ex(TA_ROWS, D, RAW16, true);
      for (long long u = u0; u < u1 && ok;) {
        const TaSeg s = ta_segment(p, plan, u, u0, u1);
        ok = mbar_wait_bounded(&q_full, n_q++ & 1, abort_v);
        for (int i = 0; i < 2 * s.n && ok; ++i) {
          int j;
          const bool is_v = ta_item(i, s.n, &j);
          ok = mbar_wait_bounded(&op_full[ring.slot], ring.phase, abort_v);
          if (ok && is_v) ok = mbar_wait_bounded(&p_full, n_p++ & 1, abort_v);
          if (!ok) break;
          tc05_fence_after();
          const uint32_t base = smem_u32(ops + ring.slot * Sh::OP);
          if (!is_v) {
            // S buffer of tile n_s: its last reader handed over P of tile n_s - 2, waited for above
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc05_mma_f16_ts(tmem + TA_S + 128 * (n_s & 1), tmem + TA_Q + 8 * kk,
                              sw128_desc(base + (kk >> 2) * (TA_TILE * 128) + (kk & 3) * 32), ID_S, kk > 0);
            tc05_commit(&s_full[n_s & 1]);
            ++n_s;
          } else {
#pragma unroll
            for (int kk = 0; kk < TA_TILE / 16; ++kk)
              tc05_mma_f16_ts(tmem + TA_O, tmem + TA_P + 8 * kk, sw128_desc_mn(base + kk * 2048, TA_TILE * 128), ID_O,
                              j > 0 || kk > 0);
            tc05_commit(&pv_done);
          }
          tc05_commit(&op_empty[ring.slot]);
          ring.next();
        }
        u += s.n;
      }
      if (!ok) {
        if (!*abort_v) raise_error(ERR_TIMEOUT_FULL);
        *abort_v = 1;
      }
      // no MMA may still be running when the tensor memory is freed: this wait
      // ignores the abort flag and ends only on completion or the time limit
      tc05_commit(&fin_bar);
      volatile int never = 0;
      mbar_wait_bounded(&fin_bar, 0, &never);
    }
  } else if (warp >= TA_SOFT) {
    // ============================================================ codes -> fp16 operands; V's odd places
    const int t = (threadIdx.x - TA_SOFT * 32) & (TA_TILE - 1), hp = (threadIdx.x - TA_SOFT * 32) / TA_TILE;
    TaRing<Sh::LOADS> in;
    TaRing<Sh::OPS> to;
    int n_seg = 0;
    bool ok = true;
    for (long long u = u0; u < u1 && ok; ++n_seg) {
      const TaSeg s = ta_segment(p, plan, u, u0, u1);
      for (int i = 0; i < 2 * s.n; ++i) {
        int j;
        const bool is_v = ta_item(i, s.n, &j);
        ok = ta_wait(&load_full[in.slot], in.phase, abort_v, ERR_TIMEOUT_FULL);
        if (!ok) break;
        const bool fix = is_v && ta_fixed(s, j);
        const int pos = (s.tile0 + j) * TA_TILE + t;
        const bool past = pos >= s.total, drafted = pos >= s.len && !past;
        bool odd = false;
        if constexpr (RAW16) {
          if (fix) {
            // Rows past the end are zeroed (their weight is 0, and 0 * NaN would not be); so are a drafted row's
            // infinities and NaN, which only rows that see it may get (added in at the end of the segment).
            if (past || drafted) {
              constexpr int CH = D / 16;                // 16-byte chunks of half a row
#pragma unroll
              for (int cc = 0; cc < CH; ++cc) {
                const int c = hp * CH + cc;             // chunk of the row, as it lies: the order does not matter here
                uint4* at = reinterpret_cast<uint4*>(ops + in.slot * Sh::OP + (c >> 3) * (TA_TILE * 128) + t * 128 + ((c & 7) << 4));
                if (past) {
                  *at = make_uint4(0, 0, 0, 0);
                } else {
                  uint4 v = *at;
                  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
                  bool hit = false;
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    if ((w[x] & 0x7f80u) == 0x7f80u) { w[x] &= 0xffff0000u; hit = true; }
                    if ((w[x] & 0x7f800000u) == 0x7f800000u) { w[x] &= 0x0000ffffu; hit = true; }
                  }
                  if (hit) { *at = v; odd = true; }
                }
              }
            }
            if (odd) s_bad[n_seg % TA_FLAGS] = 1;
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&op_full[in.slot]);
          in.next();
        } else {
          ok = ta_wait(&op_empty[to.slot], to.phase ^ 1, abort_v, ERR_TIMEOUT_EMPTY);
          if (!ok) break;
          const uint8_t* raw = raws + in.slot * Sh::RAW;
          constexpr int G = D / GROUP;
          const __half* sc = reinterpret_cast<const __half*>(raw + Sh::CODES) + t * G;
          const __half* bi = reinterpret_cast<const __half*>(raw + Sh::CODES + Sh::SIDE) + t * G;
          __half sg[G], bg[G];
          if constexpr (G == 2) {
            const uint32_t a = *reinterpret_cast<const uint32_t*>(sc), b = *reinterpret_cast<const uint32_t*>(bi);
            sg[0] = __ushort_as_half((unsigned short)a); sg[1] = __ushort_as_half((unsigned short)(a >> 16));
            bg[0] = __ushort_as_half((unsigned short)b); bg[1] = __ushort_as_half((unsigned short)(b >> 16));
          } else {
            sg[0] = sc[0];
            bg[0] = bi[0];
          }
          if (fix) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const bool wild = ta_half_bad(__half_as_ushort(sg[g])) || ta_half_bad(__half_as_ushort(bg[g]));
              if (past || (drafted && wild)) sg[g] = bg[g] = __ushort_as_half((unsigned short)0);
              odd |= drafted && wild;
            }
            if (odd) s_bad[n_seg % TA_FLAGS] = 1;
          }
          // A thread takes every other 16 bytes of its token's codes in an order that keeps 8 neighbouring lanes
          // (tokens) on 8 different bank groups, both for these loads and for the swizzled stores.
          constexpr int PARTS = D * BITS / 128, PERT = 128 / BITS;   // 16-byte parts of a row, codes in one
          const int f = PARTS == 8 ? t & 7
                        : (PARTS == 4 ? (BITS == 4 ? (t >> 1) & 3 : (((t >> 1) & 1) << 1) | (((t >> 1) ^ (t >> 2)) & 1)) : 0);
          uint8_t* row = ops + to.slot * Sh::OP + t * 128;
#pragma unroll
          for (int x = 0; x < PARTS / 2; ++x) {
            const int part = (hp * (PARTS / 2) + x) ^ f;
            const uint4 v = *reinterpret_cast<const uint4*>(raw + t * (D * BITS / 8) + part * 16);
            const int g = G == 1 ? 0 : part * PERT / GROUP;
            const __half2 s2 = __half2half2(G == 2 && g ? sg[G - 1] : sg[0]), b2 = __half2half2(G == 2 && g ? bg[G - 1] : bg[0]);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[64 / BITS];
#pragma unroll
            for (int y = 0; y < 4; ++y) ta_dequant<BITS>(w[y], s2, b2, o + y * (16 / BITS));
            uint8_t* half = row + (part * PERT / 64) * (TA_TILE * 128);
            const int c0 = part * PERT / 8 & 7;
#pragma unroll
            for (int y = 0; y < PERT / 8; ++y)
              *reinterpret_cast<uint4*>(half + (((c0 + y) ^ (t & 7)) << 4)) = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          }
          fence_proxy_async_smem();  // the tensor cores read these writes through the async proxy
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&op_full[to.slot]);
            mbar_arrive(&load_empty[in.slot]);
          }
          in.next();
          to.next();
        }
      }
      u += s.n;
    }
  } else {
    // ============================================================ softmax, and the ends of segments
    const int L = threadIdx.x;                          // tensor-memory lane
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    uint32_t n_tile = 0;                                // tiles so far: phases of s_full, pv_done
    int n_seg = 0;
    bool ok = true;
    for (long long u = u0; u < u1 && ok; ++n_seg) {
      const TaSeg s = ta_segment(p, plan, u, u0, u1);
      const int span = TA_ROWS / s.split;               // lanes of one group
      const int rr = L & (span - 1), grp = L / span;
      const bool real = rr < s.rows;
      const int r = s.rb * TA_ROWS + rr;
      const int di = real ? r / p.group : 0, hg = real ? r - di * p.group : 0;
      const int row = s.row0 + di;
      const uint64_t bits = real ? ta_mask(p, row, di, s.m) : 0;
      float f;                                          // score -> exponent of 2
      {
        uint32_t w[D / 2];
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (size_t)row * p.ldq + (s.h * p.group + hg) * D);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = real ? src[c] : make_uint4(0, 0, 0, 0);
          w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
        }
        const bool minus = p.scale < 0.f;               // the sign goes into q, so a larger S is a larger score
        f = fabsf(p.scale) * 1.4426950408889634f;
        if constexpr (RAW16) {
#pragma unroll
          for (int c = 0; c < D / 2; ++c) w[c] ^= minus ? 0x80008000u : 0u;
        } else {
          float mx = 0.f;
#pragma unroll
          for (int c = 0; c < D / 2; ++c)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[c] << 16)), fabsf(__uint_as_float(w[c] & 0xffff0000u))));
          const int ex = scale_exponent(mx);
          const float up = minus ? -pow2_exact(ex) : pow2_exact(ex);
          f *= pow2_exact(-ex);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            float x[8];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              x[2 * y] = __uint_as_float(w[4 * c + y] << 16) * up;
              x[2 * y + 1] = __uint_as_float(w[4 * c + y] & 0xffff0000u) * up;
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
              w[4 * c + y] = BITS == 4 ? ta_pack(x[y], x[y + 4], false) : ta_pack(x[2 * y], x[2 * y + 1], false);
          }
        }
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t x[32];
#pragma unroll
          for (int y = 0; y < 32; ++y) x[y] = w[32 * c + y];
          tmem_st32(tmem + TA_Q + lanes + 32 * c, x);
        }
        if (s.split > 1) {                              // the blocks of P off the diagonal
          uint32_t x[32];
#pragma unroll
          for (int y = 0; y < 32; ++y) x[y] = 0;
          tmem_st32(tmem + TA_P + lanes, x);
          tmem_st32(tmem + TA_P + lanes + 32, x);
        }
        tmem_st_wait();
        tc05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full);
      }
      float ref = -INFINITY, sum = 0.f;                 // weights are 2^(z - ref)
      const int nc = 4 / s.split, c_first = grp * nc;   // 32-token chunks of a tile for this lane
      for (int j = 0; j < s.n; ++j, ++n_tile) {
        const uint32_t sbuf = tmem + TA_S + 128 * (n_tile & 1) + lanes;
        ok = ta_wait(&s_full[n_tile & 1], (n_tile >> 1) & 1, abort_v, ERR_TIMEOUT_FULL);
        if (!ok) break;
        tc05_fence_after();
        const int t0 = (s.tile0 + j) * TA_TILE;
        const bool masked = t0 + TA_TILE > s.len;
        // visible tokens of chunk c as bits
        auto seen = [&](int c) -> uint32_t {
          const int d = t0 + 32 * c - s.len;            // drafted index of the chunk's first token
          if (d <= -32) return 0xffffffffu;
          if (d < 0) return ((1u << -d) - 1) | (uint32_t)(bits << -d);
          return d < 64 ? (uint32_t)(bits >> d) : 0u;
        };
        uint32_t v[32];
        float mx = -INFINITY;
        for (int c = c_first; c < c_first + nc; ++c) {
          tmem_ld32(sbuf + 32 * c, v);
          if (masked) {
            const uint32_t m = seen(c);
#pragma unroll
            for (int x = 0; x < 32; ++x) mx = fmaxf(mx, m >> x & 1 ? __uint_as_float(v[x]) : -INFINITY);
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) mx = fmaxf(mx, __uint_as_float(v[x]));
          }
        }
        const float top = mx == -INFINITY ? mx : mx * f;
        const bool grown = top - ref > TA_GROW;         // false for -inf - -inf
        bool waited = j == 0;
        if (__any_sync(0xffffffffu, grown)) {
          float fix = 1.f;
          if (grown) {
            const float now = top - TA_BIAS;
            fix = ta_exp2(ref - now);
            ref = now;
            sum *= fix;
          }
          if (j > 0) {
            ok = ta_wait(&pv_done, (n_tile - 1) & 1, abort_v, ERR_TIMEOUT_FULL);
            if (!ok) break;
            waited = true;
            tc05_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tmem + TA_O + lanes + 32 * c, o);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * fix);
              tmem_st32(tmem + TA_O + lanes + 32 * c, o);
            }
          }
        }
        const float sub = ref == -INFINITY ? 0.f : ref;
        if (!waited) {                                  // P is free once the product before has read it
          ok = ta_wait(&pv_done, (n_tile - 1) & 1, abort_v, ERR_TIMEOUT_FULL);
          if (!ok) break;
          tc05_fence_after();
        }
        for (int c = c_first; c < c_first + nc; ++c) {
          if (nc > 1) tmem_ld32(sbuf + 32 * c, v);
          const uint32_t m = masked ? seen(c) : 0xffffffffu;
          uint32_t w[16];
          float a0 = 0.f, a1 = 0.f;
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float e0 = ta_exp2(fmaf(__uint_as_float(v[2 * x]), f, -sub));
            float e1 = ta_exp2(fmaf(__uint_as_float(v[2 * x + 1]), f, -sub));
            if (masked) {
              e0 = m >> (2 * x) & 1 ? e0 : 0.f;
              e1 = m >> (2 * x + 1) & 1 ? e1 : 0.f;
            }
            a0 += e0;
            a1 += e1;
            w[x] = ta_pack(e0, e1, RAW16);
          }
          sum += a0 + a1;
          tmem_st16(tmem + TA_P + lanes + 16 * c, w);
        }
        tmem_st_wait();
        tc05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full);
      }
      if (ok) ok = ta_wait(&pv_done, (n_tile - 1) & 1, abort_v, ERR_TIMEOUT_FULL);
      // all four warps meet before the exchange, and go on together or not at all
      s_max[L] = ref;
      s_sum[L] = sum;
      if (lane == 0) s_ok[warp] = ok;
      named_bar_sync(1, TA_SOFT * 32);
      if (!(s_ok[0] && s_ok[1] && s_ok[2] && s_ok[3])) break;
      tc05_fence_after();
      float most = -INFINITY, weight = 0.f;
      for (int g = 0; g < s.split; ++g) most = fmaxf(most, s_max[g * span + rr]);
      const float base = most == -INFINITY ? 0.f : most;
      for (int g = 0; g < s.split; ++g) weight += s_sum[g * span + rr] * ta_exp2(s_max[g * span + rr] - base);
      const bool whole = s.n == s.nt;
      const float own = ta_exp2(ref - base);
      const float factor = whole ? (weight == 0.f ? 0.f : own / weight) : own;
      const size_t slot = 2 * (size_t)blockIdx.x + (s.first ? 0 : 1);
      if (!whole && grp == 0) {
        p.stats[(2 * slot) * TA_ROWS + rr] = most;
        p.stats[(2 * slot + 1) * TA_ROWS + rr] = weight;
      }
      const bool odd = s_bad[n_seg % TA_FLAGS] != 0;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tmem + TA_O + lanes + 32 * c, o);
        float* dst = scratch + L * TA_PAD;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          float4 q4;
          float* q = reinterpret_cast<float*>(&q4);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int d = 4 * x + y;                    // natural element; codes of 4 bits sit at another position
            const int at = BITS == 4 ? (d & ~7) + 2 * (d & 3) + ((d >> 2) & 1) : d;
            q[y] = __uint_as_float(o[at]) * factor;
          }
          *reinterpret_cast<float4*>(dst + 4 * x) = q4;
        }
        named_bar_sync(1, TA_SOFT * 32);
        const int d0 = 4 * (L & 7);
        for (int k = L >> 3; k < s.rows; k += 16) {
          float4 a = *reinterpret_cast<const float4*>(scratch + k * TA_PAD + d0);
          for (int g = 1; g < s.split; ++g) {
            const float4 b = *reinterpret_cast<const float4*>(scratch + (g * span + k) * TA_PAD + d0);
            a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
          }
          const int rk = s.rb * TA_ROWS + k, ik = rk / p.group, hk = s.h * p.group + rk - ik * p.group;
          if (odd) {                                    // rare: what was zeroed in V, for the rows that see it
            float* e = reinterpret_cast<float*>(&a);
            const uint64_t mine = ta_mask(p, s.row0 + ik, ik, s.m);
            for (int jd = 0; jd < s.m; ++jd) {
              const int pos = s.len + jd;
              if (!(mine >> jd & 1) || pos < s.tile0 * TA_TILE || pos >= (s.tile0 + s.n) * TA_TILE) continue;
              const int page = p.table[(size_t)s.b * p.table_pages + (pos >> p.c.page_shift)];
              if (page < 0 || page >= p.c.n_pages) continue;
              const size_t tok = kv_token(p.c, page, s.h, pos & ((1 << p.c.page_shift) - 1));
              for (int y = 0; y < 4; ++y) {
                const float val = ta_cache_value<BITS>(p.c.p.v, p.c.p.vs, p.c.p.vb, tok, D, 32 * c + d0 + y);
                if (!isfinite(val)) e[y] += val;
              }
            }
          }
          if (whole) {
            __nv_bfloat162 o2[2] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w)};
            *reinterpret_cast<uint2*>(p.out + (size_t)(s.row0 + ik) * p.ldo + hk * D + 32 * c + d0) = *reinterpret_cast<uint2*>(o2);
          } else {
            *reinterpret_cast<float4*>(p.partial + (slot * TA_ROWS + k) * D + 32 * c + d0) = a;
          }
        }
        named_bar_sync(1, TA_SOFT * 32);
      }
      if (L == 0) s_bad[n_seg % TA_FLAGS] = 0;
      u += s.n;
    }
  }
  tc05_fence_before();
  __syncthreads();
  if (warp == TA_MMA) {
    tc05_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial sums of items that spanned CTAs, in CTA order; a warp per (row, query head).
template <int D>
__global__ void __launch_bounds__(256) tree_attn_join_kernel(const __grid_constant__ TreeAttnParams p) {
  __shared__ TaPlan plan;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) ta_plan(p.c, p.map, p.kv_len, p.table_pages, p.group, &plan, false);
  __syncthreads();
  const int heads = p.c.heads * p.group;
  const long long id = (long long)blockIdx.x * 8 + warp;
  const int row = (int)(id / heads), hq = (int)(id - (long long)row * heads);
  if (row >= p.map.offs[p.map.B]) return;
  const int b = request_of(p.map, row), i = row - p.map.offs[b], m = p.map.offs[b + 1] - p.map.offs[b];
  const int h = hq / p.group, r = i * p.group + (hq - h * p.group), rb = r / TA_ROWS, k = r - rb * TA_ROWS;
  const int nt = (plan.len[b] + m + TA_TILE - 1) / TA_TILE;
  const long long units = plan.pre[p.map.B], per = (units + p.grid - 1) / p.grid;
  const long long a0 = plan.pre[b] + ((long long)h * ta_blocks(m, p.group) + rb) * nt;
  const int c0 = (int)(a0 / per), c1 = (int)((a0 + nt - 1) / per);
  if (c0 == c1) return;                                // one CTA had the whole item and wrote the output
  // CTA c's run of this item is its first one unless the item began inside the CTA's range
  auto slot_of = [&](int c) -> size_t { return 2 * (size_t)c + (c == c0 && a0 > (long long)c * per ? 1 : 0); };
  float most = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) most = fmaxf(most, p.stats[2 * slot_of(c) * TA_ROWS + k]);
#pragma unroll
  for (int off = 16; off; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
  const float base = most == -INFINITY ? 0.f : most;
  constexpr int E = D / 32;
  float acc[E] = {}, weight = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const size_t slot = slot_of(c);
    const float w = ta_exp2(p.stats[2 * slot * TA_ROWS + k] - base);
    weight += p.stats[(2 * slot + 1) * TA_ROWS + k] * w;
    const float* src = p.partial + (slot * TA_ROWS + k) * D + lane * E;
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
static size_t ta_partial_bytes(int grid, int dim) { return (size_t)2 * grid * TA_ROWS * dim * sizeof(float); }
static size_t ta_stats_bytes(int grid) { return (size_t)4 * grid * TA_ROWS * sizeof(float); }

template <int D, int BITS>
static cudaError_t launch_tree_attn(const TreeAttnParams& p, bool join, cudaStream_t s) {
  using Sh = TaShape<D, BITS>;
  cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<D, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(p.grid), dim3(TA_THREADS), Sh::SMEM, s, attr);
  e = cudaLaunchKernelEx(&cfg, tree_attn_kernel<D, BITS>, p);
  if (e != cudaSuccess || !join) return e;
  const long long pairs = (long long)p.map.offs[p.map.B] * p.c.heads * p.group;
  cudaLaunchConfig_t cfg2 = pdl_config(dim3((unsigned)((pairs + 7) / 8)), dim3(256), 0, s, attr);
  return cudaLaunchKernelEx(&cfg2, tree_attn_join_kernel<D>, p);
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
  // the lengths are on the device: size the grid for the longest the table allows
  const long long most_tiles = (((long long)table_pages << p.c.page_shift) + TA_TILE - 1) / TA_TILE;
  long long most = 0;
  for (int b = 0; b < B; ++b) most += (long long)p.c.heads * ta_blocks(p.map.offs[b + 1] - p.map.offs[b], p.group) * most_tiles;
  p.grid = most < sms ? (int)most : sms;
  if (p.c.bits == 16) {
    const uint64_t slabs = (uint64_t)p.c.n_pages * p.c.heads, page = 1ull << p.c.page_shift;
    const uint32_t box = page < TA_TILE ? (uint32_t)page : TA_TILE;
    st = encode_tiled_3d_sw128(&p.tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.c.p.k, p.c.dim, page, slabs, 2, 64, box);
    if (!st) st = encode_tiled_3d_sw128(&p.tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.c.p.v, p.c.dim, page, slabs, 2, 64, box);
    if (st) return st;
  }
  const bool join = most_tiles > 1;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (p.c.dim == 128)
    e = p.c.bits == 16 ? launch_tree_attn<128, 16>(p, join, s)
                       : (p.c.bits == 8 ? launch_tree_attn<128, 8>(p, join, s) : launch_tree_attn<128, 4>(p, join, s));
  else
    e = p.c.bits == 16 ? launch_tree_attn<64, 16>(p, join, s)
                       : (p.c.bits == 8 ? launch_tree_attn<64, 8>(p, join, s) : launch_tree_attn<64, 4>(p, join, s));
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "tree attention launch");
}

}  // extern "C"
