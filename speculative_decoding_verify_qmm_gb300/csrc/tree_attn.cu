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
constexpr int TA_SOFT = 4, TA_TEAM = 4;            // softmax warps (0-3); warps of a transforming team
constexpr int TA_PAD = 36;                         // floats per scratch row of 32 (16-byte aligned, conflict-free)
constexpr int TA_FLAGS = 16;                       // segments whose flags are alive at once (ring depth / 2 at most)
// tensor-memory columns
constexpr uint32_t TA_S = 0, TA_O = 256, TA_Q = 384;  // two S buffers, each overwritten by its P; O; Q
constexpr float TA_BIAS = 8.f, TA_GROW = 14.f;     // weights start at 2^8 at most and may grow to 2^14

// Warps: softmax, transforming teams, the copying warp (16-bit caches), the MMA warp.
template <int D, int BITS>
struct TaShape {
  static constexpr int TEAMS = BITS == 16 ? 1 : 3;
  static constexpr int PROD = TA_SOFT + TEAMS * TA_TEAM, MMA = PROD + 1, THREADS = (MMA + 1) * 32;
  static constexpr int OP = TA_TILE * D * 2;                                       // one operand tile, 16 bits a value
  static constexpr int SCRATCH = TA_ROWS * TA_PAD * 4;
  static constexpr int OPS = D == 128 ? 6 : 12;                                    // ring of operand tiles
  static constexpr int SMEM = 1024 + OPS * OP + SCRATCH;
  static_assert(SMEM <= 220 * 1024, "shared memory");
  static_assert(OPS % TEAMS == 0, "a team meets its slots in every turn, so it sees every phase of their barriers");
  static_assert(OPS <= 2 * TA_FLAGS - 4, "flags");
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

// One operand tile of codes as the transforming warps need it: the cache's token index of each 16 tokens (-1: past the
// end), and what is odd about it.
struct TaPiece {
  long long tok[TA_TILE / 16];
  long long valid;              // tokens of the tile before the end of the sequence
  long long drafted;            // first drafted token of the tile (TA_TILE and more: none)
  long long is_v;
  long long flag;               // the segment's flag in s_bad
};
constexpr int TA_PIECES = 12;   // descriptors in flight

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
// 16 bytes that are read once: kept out of L1.
__device__ __forceinline__ uint4 ld_stream16(const uint8_t* a) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(a));
  return v;
}
__device__ __forceinline__ bool ta_half_bad(uint32_t h) { return (h & 0x7c00u) == 0x7c00u; }

__device__ __forceinline__ float ta_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max of three (NaN operands are passed over, as by fmaxf)
__device__ __forceinline__ float ta_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

// mbar_wait_bounded that looks at the clock (a slow read) only after some polls.
__device__ __forceinline__ bool ta_poll(uint64_t* bar, uint32_t parity, volatile int* abort_v) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait_bounded(bar, parity, abort_v);
}
// A whole warp waits; false for all lanes once any gave up (the reason is recorded once).
__device__ __forceinline__ bool ta_wait(uint64_t* bar, uint32_t parity, volatile int* abort_v, unsigned err) {
  bool ok = ta_poll(bar, parity, abort_v);
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
__global__ void __launch_bounds__(TaShape<D, BITS>::THREADS, 1) tree_attn_kernel(const __grid_constant__ TreeAttnParams p) {
  using Sh = TaShape<D, BITS>;
  constexpr bool RAW16 = BITS == 16;
  extern __shared__ uint8_t smem_raw[];
  // operand slots: copied into (16-bit caches only), ready for the tensor cores, read
  __shared__ uint64_t load_full[Sh::OPS], op_full[Sh::OPS], op_empty[Sh::OPS];
  __shared__ uint64_t q_full, s_full[2], p_full[2], pv_done, fin_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int abort_flag, s_bad[TA_FLAGS];
  __shared__ TaPlan plan;
  __shared__ TaPiece pieces[RAW16 ? 1 : TA_PIECES];     // caches of codes: filled by the copying warp, read by one team each
  __shared__ uint64_t piece_full[TA_PIECES], piece_empty[TA_PIECES];
  __shared__ float s_max[TA_ROWS], s_sum[TA_ROWS];
  __shared__ int s_ok[TA_SOFT];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const ops = smem;
  float* const scratch = reinterpret_cast<float*>(smem + Sh::OPS * Sh::OP);
  volatile int* abort_v = &abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::OPS; ++i) {
      mbar_init(&load_full[i], 1);
      mbar_init(&op_full[i], TA_TEAM);
      mbar_init(&op_empty[i], 1);
    }
    for (int i = 0; i < TA_PIECES; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], TA_TEAM);
    }
    mbar_init(&q_full, TA_SOFT);
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(&p_full[0], TA_SOFT);
    mbar_init(&p_full[1], TA_SOFT);
    mbar_init(&pv_done, 1);
    mbar_init(&fin_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < TA_FLAGS) s_bad[threadIdx.x] = 0;
  if (warp == Sh::MMA) {
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

  if (warp == Sh::PROD) {
    // ============================================================ copies of a 16-bit cache into the ring
    if constexpr (RAW16) {
      const int shift = p.c.page_shift < 7 ? p.c.page_shift : 7, chunk = 1 << shift;   // tokens per copy
      const int place_mask = (1 << p.c.page_shift) - 1;
      constexpr int PER = D / 64;                      // copies per chunk: 64-wide pieces of the head
      const int my_chunk = lane / PER, part = lane - my_chunk * PER;
      TaRing<Sh::OPS> ring;
      bool ok = true;
      for (long long u = u0; u < u1 && ok;) {
        const TaSeg s = ta_segment(p, plan, u, u0, u1);
        // the table's entry for this lane's chunk of tile j, checked when it is used: the load is a tile ahead
        auto page_of = [&](int j) -> int {
          const int t = (s.tile0 + j) * TA_TILE + (my_chunk << shift);
          if (j >= s.n || my_chunk >= (TA_TILE >> shift) || t >= s.total) return 0;
          return p.table[(size_t)s.b * p.table_pages + (t >> p.c.page_shift)];
        };
        int page_before = 0, page_k = 0, page_next = page_of(0);   // of the last two K tiles, and the next one's
        for (int i = 0; i < 2 * s.n; ++i) {
          int j;
          const bool is_v = ta_item(i, s.n, &j);
          if (!is_v) {
            page_before = page_k;
            page_k = page_next;
            page_next = page_of(j + 1);
          }
          int page = is_v && i != 2 * s.n - 1 ? page_before : page_k;
          ok = ta_wait(&op_empty[ring.slot], ring.phase ^ 1, abort_v, ERR_TIMEOUT_EMPTY);
          if (!ok) break;
          const int t0 = (s.tile0 + j) * TA_TILE;
          const int toks = s.total - t0 < TA_TILE ? s.total - t0 : TA_TILE;
          const int chunks = (toks + chunk - 1) >> shift;
          if (lane == 0) mbar_arrive_expect_tx(&load_full[ring.slot], (uint32_t)(chunks << shift) * (D * 2));
          __syncwarp();
          if (my_chunk < chunks) {
            if (page < 0 || page >= p.c.n_pages) {
              raise_error(ERR_BAD_INPUT);
              page = 0;                                // stay inside the arrays: the result is undefined
            }
            const int place = (t0 + (my_chunk << shift)) & place_mask;
            uint8_t* dst = ops + ring.slot * Sh::OP + part * (TA_TILE * 128) + (my_chunk << shift) * 128;
            tma_load_3d_plain(dst, is_v ? &p.tv : &p.tk, &load_full[ring.slot], part * 64, place, page * p.c.heads + s.h);
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
    } else {
      // ========================================================== descriptors for the transforming warps
      TaRing<TA_PIECES> ring;
      const int pm = (1 << p.c.page_shift) - 1;
      int n_seg = 0;
      bool ok = true;
      for (long long u = u0; u < u1 && ok; ++n_seg) {
        const TaSeg s = ta_segment(p, plan, u, u0, u1);
        auto page_of = [&](int j) -> int {             // of 16-token piece `lane` of tile j; checked when it is used
          const int t = (s.tile0 + j) * TA_TILE + 16 * lane;
          if (j >= s.n || lane >= TA_TILE / 16 || t >= s.total) return 0;
          return p.table[(size_t)s.b * p.table_pages + (t >> p.c.page_shift)];
        };
        int page_before = 0, page_k = 0, page_next = page_of(0);   // of the last two K tiles, and the next one's
        for (int i = 0; i < 2 * s.n; ++i) {
          int j;
          const bool is_v = ta_item(i, s.n, &j);
          if (!is_v) {
            page_before = page_k;
            page_k = page_next;
            page_next = page_of(j + 1);
          }
          int page = is_v && i != 2 * s.n - 1 ? page_before : page_k;
          ok = ta_wait(&piece_empty[ring.slot], ring.phase ^ 1, abort_v, ERR_TIMEOUT_EMPTY);
          if (!ok) break;
          const int t0 = (s.tile0 + j) * TA_TILE, t = t0 + 16 * lane;
          if ((unsigned)page >= (unsigned)p.c.n_pages) {
            raise_error(ERR_BAD_INPUT);
            page = 0;                                  // stay inside the arrays: the result is undefined
          }
          // one store for the whole descriptor: lane i writes its i-th word
          long long word = t < s.total ? (long long)kv_token(p.c, page, s.h, t & pm) : -1;
          word = lane == 8 ? s.total - t0 : (lane == 9 ? s.len - t0 : word);
          word = lane == 10 ? (long long)is_v : (lane == 11 ? n_seg % TA_FLAGS : word);
          if (lane < (int)(sizeof(TaPiece) / 8)) reinterpret_cast<long long*>(&pieces[ring.slot])[lane] = word;
          __syncwarp();
          if (lane == 0) mbar_arrive(&piece_full[ring.slot]);
          ring.next();
        }
        u += s.n;
      }
      // the end: one descriptor for each team
      for (int e = 0; e < Sh::TEAMS && ok; ++e) {
        ok = ta_wait(&piece_empty[ring.slot], ring.phase ^ 1, abort_v, ERR_TIMEOUT_EMPTY);
        if (!ok) break;
        if (lane < TA_TILE / 16) pieces[ring.slot].tok[lane] = -1;
        if (lane == 8) pieces[ring.slot].valid = 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&piece_full[ring.slot]);
        ring.next();
      }
    }
  } else if (warp == Sh::MMA) {
    // ============================================================ MMA issue
    // The whole warp runs the loop and one lane issues, so that descriptors and addresses live in uniform registers.
    {
      TaRing<Sh::OPS> ring;
      uint32_t n_q = 0, n_s = 0, n_p = 0;               // phases seen of each barrier
      bool ok = true;
      constexpr uint32_t ID_S = f16_idesc_ex(TA_ROWS, TA_TILE, RAW16, false);
      constexpr uint32_t ID_O = f16_idesc_ex(TA_ROWS, D, RAW16, true);
      const bool issuer = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t ops0 = (__shfl_sync(0xffffffffu, smem_u32(ops), 0) & 0x3FFFFu) >> 4;
      // descriptors differ in the start address alone
      constexpr uint32_t HI = (1024u >> 4) | (1u << 14) | (2u << 29);
      constexpr uint32_t LO_K = 1u << 16, LO_V = (uint32_t)(TA_TILE * 128 >> 4) << 16;
      for (long long u = u0; u < u1 && ok;) {
        int n;
        {
          const TaSeg s = ta_segment(p, plan, u, u0, u1);
          n = __shfl_sync(0xffffffffu, s.n, 0);
        }
        ok = ta_wait(&q_full, n_q++ & 1, abort_v, ERR_TIMEOUT_FULL);
        for (int i = 0; i < 2 * n && ok; ++i) {
          const bool is_v = i == 2 * n - 1 || (i > 0 && !(i & 1));
          ok = ta_wait(&op_full[ring.slot], ring.phase, abort_v, ERR_TIMEOUT_FULL);
          if (ok && is_v) ok = ta_wait(&p_full[n_p & 1], (n_p >> 1) & 1, abort_v, ERR_TIMEOUT_FULL);
          if (!ok) break;
          tc05_fence_after();
          const uint32_t base = ops0 + ring.slot * (Sh::OP >> 4);
          if (!is_v) {
            // S buffer of tile n_s: P of tile n_s - 2 lies there, whose product was issued before (MMAs run in order)
            const uint32_t d = tm + TA_S + 128 * (n_s & 1), lo = base | LO_K;
            if (issuer) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc05_mma_f16_ts(d, tm + TA_Q + 8 * kk, lo + (kk >> 2) * (TA_TILE * 128 >> 4) + (kk & 3) * 2, HI, ID_S, kk > 0);
              tc05_commit(&s_full[n_s & 1]);
              tc05_commit(&op_empty[ring.slot]);
            }
            ++n_s;
          } else {
            const uint32_t a = tm + TA_S + 128 * (n_p & 1), lo = base | LO_V;
            const bool first = i < 3 && !(i == 1 && n > 1);   // V of the segment's first tile: item 2, or 1 of 2
            if (issuer) {
#pragma unroll
              for (int kk = 0; kk < TA_TILE / 16; ++kk)
                tc05_mma_f16_ts(tm + TA_O, a + 8 * kk, lo + kk * (2048 >> 4), HI, ID_O, !first || kk > 0);
              tc05_commit(&pv_done);
              tc05_commit(&op_empty[ring.slot]);
            }
            ++n_p;
          }
          __syncwarp();
          ring.next();
        }
        u += n;
      }
      // no MMA may still be running when the tensor memory is freed: this wait
      // ignores the abort flag and ends only on completion or the time limit
      if (issuer) {
        tc05_commit(&fin_bar);
        volatile int never = 0;
        mbar_wait_bounded(&fin_bar, 0, &never);
      }
      __syncwarp();
    }
  } else if (warp >= TA_SOFT) {
    const int team = (warp - TA_SOFT) / TA_TEAM, tw = (warp - TA_SOFT) % TA_TEAM;
    const int t = 32 * tw + lane;                       // this lane's token of a tile
    if constexpr (RAW16) {
      // ========================================================== a 16-bit cache: V's odd places
      TaRing<Sh::OPS> ring;
      int n_seg = 0;
      bool ok = true;
      for (long long u = u0; u < u1 && ok; ++n_seg) {
        const TaSeg s = ta_segment(p, plan, u, u0, u1);
        for (int i = 0; i < 2 * s.n; ++i, ring.next()) {
          int j;
          const bool is_v = ta_item(i, s.n, &j);
          ok = ta_wait(&load_full[ring.slot], ring.phase, abort_v, ERR_TIMEOUT_FULL);
          if (!ok) break;
          const int pos = (s.tile0 + j) * TA_TILE + t;
          if (is_v && ta_fixed(s, j)) {
            // Rows past the end are zeroed (their weight is 0, and 0 * NaN would not be); so are a drafted row's
            // infinities and NaN, which only rows that see it may get (added in at the end of the segment).
            if (pos >= s.len) {
              const bool past = pos >= s.total;
              bool odd = false;
#pragma unroll
              for (int c = 0; c < D / 8; ++c) {         // chunks of the row as they lie: the order does not matter here
                uint4* at = reinterpret_cast<uint4*>(ops + ring.slot * Sh::OP + (c >> 3) * (TA_TILE * 128) + t * 128 + ((c & 7) << 4));
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
              if (odd) s_bad[n_seg % TA_FLAGS] = 1;
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&op_full[ring.slot]);
        }
        u += s.n;
      }
    } else {
      // ========================================================== codes -> fp16 operands
      // A team takes every third operand tile, a warp 32 of its tokens.  Codes come from global memory in 16-byte
      // loads, LPT neighbouring lanes per token; the registers of a step are loaded for the team's next tile as soon
      // as they are used, so the loads of a whole tile are always on their way.
      constexpr int ROWB = D * BITS / 8, LPT = ROWB / 16, TPS = 32 / LPT, PERT = 128 / BITS;  // codes per 16 bytes
      constexpr int NCH = PERT / 8, G = D / GROUP;      // 16-byte operand chunks a lane makes per step; groups per token
      const int part = lane & (LPT - 1), sub = lane / LPT;
      const int grp = part * PERT / GROUP, c0 = (part * PERT / 8) & 7;
      // Which of its chunks a lane stores first, so that 8 neighbouring lanes meet 8 different bank groups.
      const int sel = LPT == 8 ? part >> 2 : (NCH == 4 && LPT == 4 ? (part >> 1) | ((sub & 1) << 1) : 0);
      const uint32_t pick = G == 2 && grp ? 0x3232 : 0x1010;
      uint8_t* const mine = ops + (part * PERT / 64) * (TA_TILE * 128) + (32 * tw + sub) * 128;
      TaRing<Sh::OPS> ring;
      TaRing<TA_PIECES> ahead, here;
      for (int i = 0; i < team; ++i) {
        ring.next();
        ahead.next();
        here.next();
      }
      uint4 raw[LPT];
      uint32_t sc = 0, bi = 0;                          // scales and biases of this lane's token (two groups, or one)
      const uint8_t* at[2] = {};                        // the warp's two 16-token halves (null: past the end)
      bool live = true;
      // the next tile's addresses, scales and biases
      auto locate = [&]() -> bool {
        if (!ta_wait(&piece_full[ahead.slot], ahead.phase, abort_v, ERR_TIMEOUT_FULL)) return false;
        const TaPiece& x = pieces[ahead.slot];
        sc = bi = 0;
        const int valid = (int)x.valid;
        live = valid > 0;
        const bool is_v = x.is_v;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const long long tok = x.tok[2 * tw + hf];
          at[hf] = tok < 0 ? nullptr : (is_v ? p.c.p.v : p.c.p.k) + tok * ROWB + lane * 16;
          if (tok >= 0 && lane / 16 == hf && t < valid) {
            const size_t g = ((size_t)tok + (lane & 15)) * G;
            const __half *ps = (is_v ? p.c.p.vs : p.c.p.ks) + g, *pb = (is_v ? p.c.p.vb : p.c.p.kb) + g;
            if constexpr (G == 2) {
              sc = *reinterpret_cast<const uint32_t*>(ps);
              bi = *reinterpret_cast<const uint32_t*>(pb);
            } else {
              sc = *reinterpret_cast<const unsigned short*>(ps);
              bi = *reinterpret_cast<const unsigned short*>(pb);
            }
          }
        }
        for (int i = 0; i < Sh::TEAMS; ++i) ahead.next();
        return true;
      };
      auto fetch = [&](int i) {
        const int hf = i * TPS / 16;
        if (at[hf]) raw[i] = ld_stream16(at[hf] + (i * TPS - 16 * hf) * ROWB);
      };
#pragma unroll
      for (int i = 0; i < LPT; ++i) raw[i] = make_uint4(0, 0, 0, 0);
      bool ok = locate();
      if (ok) {
#pragma unroll
        for (int i = 0; i < LPT; ++i) fetch(i);
      }
      while (ok && live) {
        uint32_t sv = sc, bv = bi;
        ok = ta_wait(&op_empty[ring.slot], ring.phase ^ 1, abort_v, ERR_TIMEOUT_EMPTY);
        if (!ok) break;
        const TaPiece& x = pieces[here.slot];
        if (x.is_v && x.drafted < TA_TILE) {
          // A V row past the end becomes zero (its weight is 0, and 0 * NaN would not be); so does a drafted row's
          // group that reads as NaN, which only rows that see it may get (added in at the end of the segment).
          const bool past = t >= x.valid, drafted = t >= x.drafted && !past;
          bool odd = false;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const bool wild = ta_half_bad(sv >> (16 * g)) || ta_half_bad(bv >> (16 * g));
            if (past || (drafted && wild)) {
              sv &= ~(0xffffu << (16 * g));
              bv &= ~(0xffffu << (16 * g));
            }
            odd |= drafted && wild;
          }
          if (odd) s_bad[x.flag] = 1;
        }
        uint8_t* const dst = mine + ring.slot * Sh::OP;
#pragma unroll
        for (int i = 0; i < LPT; ++i) {
          uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          const uint32_t s1 = __shfl_sync(0xffffffffu, sv, i * TPS + sub), b1 = __shfl_sync(0xffffffffu, bv, i * TPS + sub);
          const uint32_t sp = __byte_perm(s1, 0, pick), bp = __byte_perm(b1, 0, pick);
          const __half2 s2 = *reinterpret_cast<const __half2*>(&sp), b2 = *reinterpret_cast<const __half2*>(&bp);
          // chunk y comes from the words of chunk y ^ sel
          if constexpr (NCH == 4 && LPT == 4) {
            if (sel & 1) { const uint32_t a = w[0], b = w[2]; w[0] = w[1]; w[1] = a; w[2] = w[3]; w[3] = b; }
          }
          if constexpr (LPT == 8 || (NCH == 4 && LPT == 4)) {
            if (sel & (NCH / 2)) { const uint32_t a = w[0], b = w[1]; w[0] = w[2]; w[2] = a; w[1] = w[3]; w[3] = b; }
          }
          uint32_t o[64 / BITS];
#pragma unroll
          for (int y = 0; y < 4; ++y) ta_dequant<BITS>(w[y], s2, b2, o + y * (16 / BITS));
          const int xr = (i * TPS + sub) & 7;           // the token's row in its swizzle group
#pragma unroll
          for (int y = 0; y < NCH; ++y)
            *reinterpret_cast<uint4*>(dst + i * TPS * 128 + (((c0 + (y ^ sel)) ^ xr) << 4)) =
                make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
        }
        fence_proxy_async_smem();  // the tensor cores read these writes through the async proxy
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&op_full[ring.slot]);
          mbar_arrive(&piece_empty[here.slot]);
        }
        for (int i = 0; i < Sh::TEAMS; ++i) {
          ring.next();
          here.next();
        }
        ok = locate();
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < LPT; ++i) fetch(i);
      }
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
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (size_t)row * p.ldq + (s.h * p.group + hg) * D);
        const bool minus = p.scale < 0.f;               // the sign goes into q, so a larger S is a larger score
        f = fabsf(p.scale) * 1.4426950408889634f;
        float up = minus ? -1.f : 1.f;
        if constexpr (!RAW16) {
          float mx = 0.f;
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = real ? src[c] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; ++y)
              mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[y] << 16)), fabsf(__uint_as_float(w[y] & 0xffff0000u))));
          }
          const int ex = scale_exponent(mx);
          up *= pow2_exact(ex);
          f *= pow2_exact(-ex);
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[16];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const uint4 v = real ? src[4 * c + z] : make_uint4(0, 0, 0, 0);
            x[4 * z] = v.x; x[4 * z + 1] = v.y; x[4 * z + 2] = v.z; x[4 * z + 3] = v.w;
          }
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            if constexpr (RAW16) {
#pragma unroll
              for (int y = 0; y < 4; ++y) x[4 * z + y] ^= minus ? 0x80008000u : 0u;
            } else {
              float e[8];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                e[2 * y] = __uint_as_float(x[4 * z + y] << 16) * up;
                e[2 * y + 1] = __uint_as_float(x[4 * z + y] & 0xffff0000u) * up;
              }
#pragma unroll
              for (int y = 0; y < 4; ++y)
                x[4 * z + y] = BITS == 4 ? ta_pack(e[y], e[y + 4], false) : ta_pack(e[2 * y], e[2 * y + 1], false);
            }
          }
          tmem_st16(tmem + TA_Q + lanes + 16 * c, x);
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
            for (int x = 0; x < 32; x += 2) mx = ta_max3(mx, __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
          }
        }
        const float top = mx == -INFINITY ? mx : mx * f;
        const bool grown = top - ref > TA_GROW;         // false for -inf - -inf
        if (__any_sync(0xffffffffu, grown)) {
          float fix = 1.f;
          if (grown) {
            const float now = top - TA_BIAS;
            fix = ta_exp2(ref - now);
            ref = now;
            sum *= fix;
          }
          if (j > 0) {
            // S of this tile is there, so the product before the last has ended: one phase is open at most
            ok = ta_wait(&pv_done, (n_tile - 1) & 1, abort_v, ERR_TIMEOUT_FULL);
            if (!ok) break;
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
        // P takes the place of S, column by column behind the reads
        for (int c = c_first; c < c_first + nc; ++c) {
          if (nc > 1) tmem_ld32(sbuf + 32 * c, v);
          const uint32_t m = masked ? seen(c) : 0xffffffffu;
          uint32_t w[16];
          float2 acc = make_float2(0.f, 0.f);
          const float2 f2 = make_float2(f, f), n2 = make_float2(-sub, -sub);
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float2 z = __ffma2_rn(make_float2(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1])), f2, n2);
            float2 e = make_float2(ta_exp2(z.x), ta_exp2(z.y));
            if (masked) {
              e.x = m >> (2 * x) & 1 ? e.x : 0.f;
              e.y = m >> (2 * x + 1) & 1 ? e.y : 0.f;
            }
            acc = __fadd2_rn(acc, e);
            w[x] = ta_pack(e.x, e.y, RAW16);
          }
          sum += acc.x + acc.y;
          tmem_st16(sbuf + 16 * c, w);
        }
        if (s.split > 1) {                              // the blocks of P off the diagonal
          const uint32_t zero[16] = {};
          for (int c = 0; c < 4; ++c)
            if (c < c_first || c >= c_first + nc) tmem_st16(sbuf + 16 * c, zero);
        }
        tmem_st_wait();
        tc05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[n_tile & 1]);
      }
      // the last product; the one before may be out too, and each phase has to be seen
      if (ok) ok = ta_wait(&pv_done, (n_tile - 2) & 1, abort_v, ERR_TIMEOUT_FULL);
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
  if (warp == Sh::MMA) {
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
  cudaLaunchConfig_t cfg = pdl_config(dim3(p.grid), dim3(Sh::THREADS), Sh::SMEM, s, attr);
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
