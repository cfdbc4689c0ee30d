// Tree attention of more than 32 rows (drafted rows x query heads per key head), on the 5th-generation tensor cores
// (mlx-dspark wiki page, "Architecture": the target verifies the drafted block in one forward over its cache).
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - max)
//
// The rows are the 128 lanes of one matrix (more: several items); the cache is streamed past them in tiles of 128 tokens.
// Per tile, S = Q K^T with Q (A operand) resident in tensor memory, K from shared memory, S [row x token] in tensor memory;
// softmax of a lane by one thread; P (16 bits) in S's place as the A operand of O += P V, V from shared memory as it lies
// ([token][element], MN-major).  O stays in tensor memory.  A row's weights are 2^(S f - ref) with a reference that moves
// only when a score has outgrown it by 2^10 (fp16) or 2^15 (bf16): rarely, and then O and what there is of P are rescaled.
//
// Up to 64 rows are laid into the lanes twice, and each copy takes its own half of every tile's tokens - the off-diagonal
// blocks of P are zero - as an independent softmax that meets the other at the end of the item: all four softmax warps
// share the work of two, without talking to each other.
//
// Bound by memory: a token costs D * bits / 4 bytes against 4 * rows * D operations, and the tensor cores see the same
// 128-row instruction however few rows are real.  16-bit caches go from TMA to the tensor cores untouched.  Codes are
// dequantized by three teams of four warps into fp16 in the operand layout, fp16(s * c + b) with the exact code (half an
// fp16 step), and Q enters as fp16 scaled by a power of two per row, exact for every bf16 value within 2^29 of the
// row's largest.
//
// Measured (8 key heads of 128): a 32-node tree in 32 heads over 65536 tokens, bf16, 60.3 us (4.5 TB/s; 46 us while tiles run, at
// the copy rate, the rest is the start, the exchange at the end and the join); 4 x 8 rows in 48 heads over up to 30001
// tokens, 8-bit, 54.4 us (3.4 TB/s).  Over codes the softmax warps set the pace, some 2500 cycles a tile beside the transforming
// warps, whose issue slots they share.
//
// Over codes, copies to shared memory ahead of the transformation were slower than loads straight to registers: 24 bulk copies a
// tile 104 us, cp.async by one warp 79 us, by the transforming warps 63.5 us, against 55.6.
//
// Tried instead: tokens and elements as lanes and rows as columns of the products (their cost then follows the rows, no
// exchange at the end, the weights' sums from a product with ones).  It needs Q and P in shared memory, which leaves three
// slots to the ring, and an instruction takes its warp some 70 cycles to issue whatever its width: 68 us against 58 for 128
// rows over 65536 tokens of a bf16 cache.
#include <type_traits>

#include "tree_attn_tc.cuh"

namespace sv {

constexpr int TA_ROWS = 128;                       // rows per block: the lanes of tensor memory
constexpr int TA_SOFT = 4;                         // softmax warps (0-3)
constexpr int TA_PAD = 36;                         // floats per scratch row of 32 (16-byte aligned, conflict-free)
constexpr int TA_FLAGS = 16;                       // segments whose flags are alive at once (ring depth / 2 at most)
// tensor-memory columns
constexpr uint32_t TA_S = 0, TA_O = 256, TA_Q = 384;  // two S buffers, each overwritten by its P; O; Q

// Warps: softmax, transforming teams, the copying warp (16-bit caches), the MMA warp.
template <int D, int BITS>
struct TaShape {
  static constexpr int TEAMS = BITS == 16 ? 1 : 3;
  static constexpr int PROD = TA_SOFT + TEAMS * TA_TEAM, MMA = PROD + 1, THREADS = (MMA + 1) * 32;
  static constexpr int OP = TA_TILE * D * 2;                                       // one operand tile, 16 bits a value
  static constexpr int SCRATCH = TA_ROWS * TA_PAD * 4;
  static constexpr int OPS = (BITS == 16 ? 6 : 3) * (128 / D);                     // ring of operand tiles (codes, 6 of them: 57.2 us against 55.6)
  static constexpr int SMEM = 1024 + OPS * OP + SCRATCH;
  static_assert(SMEM <= 220 * 1024, "shared memory");
  static_assert(OPS % TEAMS == 0, "a team meets its slots in every turn, so it sees every phase of their barriers");
  static_assert(OPS <= 2 * TA_FLAGS - 4, "flags");
  // A weight enters the second product in 16 bits.  BIAS: exponent of the largest weight when the reference is set, GROW: what
  // it may grow to before the reference moves.  fp16 has room up to 2^15; there the largest weight starts at 2^5, so that weights
  // down to 2^-19 of it keep all their bits and smaller ones are off by at most 2^-30 of it (2^20 such tokens: 2^-10 of their values;
  // a higher start would move the reference, and rescale, more often).  bf16 has the range of fp32, and so have the values of a
  // 16-bit cache: weights of at most 2^-15 keep the sums of any finite values finite (of 2^15 tokens at GROW, of 2^30 at BIAS), and
  // at BIAS those down to 2^-96 of the largest keep all their bits.
  static constexpr float BIAS = BITS == 16 ? -30.f : 5.f, GROW = BITS == 16 ? -15.f : 15.f;
};

// Order of a segment's operand tiles: K0, K1, V0, K2, V1, ..., V(n-1).
__device__ __forceinline__ bool ta_item(int e, int n, int* tile) {
  if (e == 0) { *tile = 0; return false; }
  if (e == 2 * n - 1) { *tile = n - 1; return true; }
  if (e & 1) { *tile = (e + 1) / 2; return false; }
  *tile = e / 2 - 1;
  return true;
}

// Tiles whose V the transforming warps look through: those with drafted tokens or past the end.
__device__ __forceinline__ bool ta_fixed(const TaSeg& s, int j) { return (s.tile0 + j + 1) * TA_TILE > s.len; }

template <int D, int BITS, typename P>
__global__ void __launch_bounds__(TaShape<D, BITS>::THREADS, 1) tree_attn_wide_kernel(const __grid_constant__ P p) {
  using Sh = TaShape<D, BITS>;
  constexpr bool RAW16 = BITS == 16;
  extern __shared__ uint8_t smem_raw[];
  // operand slots: copied into (16-bit caches only), ready for the tensor cores, read
  __shared__ uint64_t load_full[Sh::OPS], op_full[Sh::OPS], op_empty[Sh::OPS];
  __shared__ uint64_t q_full, s_full[2], p_full[2], pv_done, run_done, fin_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int abort_flag, s_bad[TA_FLAGS];
  __shared__ TaPlan plan;
  __shared__ TaPiece pieces[RAW16 ? 1 : TA_PIECES];     // caches of codes: filled by the copying warp, read by one team each
  __shared__ uint64_t piece_full[TA_PIECES], piece_empty[TA_PIECES];
  __shared__ float s_max[TA_ROWS], s_sum[TA_ROWS];
  __shared__ int s_ok[TA_SOFT];
  __shared__ long long s_out[TA_ROWS];                   // where each row of the block is written (elements)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const ops = smem;
  float* const scratch = reinterpret_cast<float*>(smem + Sh::OPS * Sh::OP);
  volatile int* abort_v = &abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
    mbar_init(&run_done, 1);
    mbar_init(&fin_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < TA_FLAGS) s_bad[threadIdx.x] = 0;
  if (warp == Sh::MMA) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  const TaShare share = ta_begin(p, &plan);
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  const uint32_t tmem = s_tmem;
  const long long u0 = share.u0, u1 = share.u1;

  if (warp == Sh::PROD) {
    // ============================================================ copies of a 16-bit cache into the ring
    if constexpr (RAW16) {
      const int shift = p.c.page_shift < 7 ? p.c.page_shift : 7, chunk = 1 << shift;   // tokens per copy
      const int place_mask = (1 << p.c.page_shift) - 1;
      constexpr int PER = D / 64;                      // copies per chunk: 64-wide pieces of the head
      const int my_chunk = lane / PER, part = lane - my_chunk * PER;
      TaRing<Sh::OPS> ring;
      bool ok = true;
      TaSeg s = share.s;
      long long u = share.u;
      for (bool more = share.more; ok && more; more = ta_next(p, plan, &u, u0, u1, &s)) {
        // the table's entry for this lane's chunk of tile j, checked when it is used: the load is a tile ahead
        auto page_of = [&](int j) -> int {
          const int t = (s.tile0 + j) * TA_TILE + (my_chunk << shift);
          if (j >= s.n || my_chunk >= (TA_TILE >> shift) || t >= s.total) return 0;
          return ta_table(p, s.b)[t >> p.c.page_shift];
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
      }
    } else {
      // ========================================================== descriptors for the transforming warps
      TaRing<TA_PIECES> ring;
      const int pm = (1 << p.c.page_shift) - 1;
      int n_seg = 0;
      bool ok = true;
      TaSeg s = share.s;
      long long u = share.u;
      for (bool more = share.more; ok && more; more = ta_next(p, plan, &u, u0, u1, &s), ++n_seg) {
        auto page_of = [&](int j) -> int {             // of 16-token piece `lane` of tile j; checked when it is used
          const int t = (s.tile0 + j) * TA_TILE + 16 * lane;
          if (j >= s.n || lane >= TA_TILE / 16 || t >= s.total) return 0;
          return ta_table(p, s.b)[t >> p.c.page_shift];
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
          TaPiece& x = pieces[ring.slot];
          if (lane < TA_TILE / 16) {
            const size_t tok = t < s.total ? kv_token(p.c, page, s.h, t & pm) : 0;
            x.codes[lane] = (is_v ? p.c.p.v : p.c.p.k) + tok * (D * BITS / 8);
            x.scales[lane] = (is_v ? p.c.p.vs : p.c.p.ks) + tok * (D / GROUP);
            x.biases[lane] = (is_v ? p.c.p.vb : p.c.p.kb) + tok * (D / GROUP);
          }
          if (lane == 8) {
            x.valid = s.total - t0;
            x.drafted = s.len - t0;
            x.is_v = is_v;
            x.flag = n_seg % TA_FLAGS;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&piece_full[ring.slot]);
          ring.next();
        }
      }
      // the end: one descriptor for each team
      for (int e = 0; e < Sh::TEAMS && ok; ++e) {
        ok = ta_wait(&piece_empty[ring.slot], ring.phase ^ 1, abort_v, ERR_TIMEOUT_EMPTY);
        if (!ok) break;
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
      TaSeg s = share.s;
      long long u = share.u;
      for (bool more = share.more; ok && more; more = ta_next(p, plan, &u, u0, u1, &s)) {
        const int n = __shfl_sync(0xffffffffu, s.n, 0);
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
              if (i == 2 * n - 1) tc05_commit(&run_done);
              tc05_commit(&op_empty[ring.slot]);
            }
            ++n_p;
          }
          __syncwarp();
          ring.next();
        }
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
      TaSeg s = share.s;
      long long u = share.u;
      for (bool more = share.more; ok && more; more = ta_next(p, plan, &u, u0, u1, &s), ++n_seg) {
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
      }
    } else {
      // ========================================================== codes -> fp16 operands
      ta_transform<D, BITS, Sh::TEAMS, Sh::OPS, true>(ops, op_full, op_empty, pieces, piece_full, piece_empty, s_bad, abort_v, team, tw, lane);
    }
  } else {
    // ============================================================ softmax, and the ends of segments
    const int L = threadIdx.x;                          // tensor-memory lane
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    uint32_t n_tile = 0;                                // tiles so far: phases of s_full, pv_done
    int n_seg = 0;
    bool ok = true;
    TaSeg s = share.s;
    long long u = share.u;
    for (bool more = share.more; ok && more; more = ta_next(p, plan, &u, u0, u1, &s), ++n_seg) {
      const int split = s.rows <= 64 ? 2 : 1;           // copies of the rows in the lanes
      const int span = TA_ROWS / split;               // lanes of one group
      const int rr = L & (span - 1), grp = L / span;
      const bool real = rr < s.rows;
      const int r = s.rb * p.block + rr;
      const int di = real ? ta_by_group(p, r) : 0, hg = real ? r - di * p.group : 0;
      const int row = s.row0 + di;
      const uint64_t bits = real ? ta_mask(p, row, di, s.m) : 0;
      float f;                                          // score -> exponent of 2
      {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (size_t)row * p.ldq + (s.h * p.group + hg) * D);
        const bool minus = p.scale < 0.f;               // the sign goes into q, so a larger S is a larger score
        f = ta_score_factor(p.scale, 0);
        float up = minus ? -1.f : 1.f;
        if constexpr (!RAW16) {
          float mx = 0.f;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = real ? src[c] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; ++y)
              mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[y] << 16)), fabsf(__uint_as_float(w[y] & 0xffff0000u))));
          }
          const int ex = ta_query_exponent(mx);
          up *= pow2_exact(ex);
          f = ta_score_factor(p.scale, ex);
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
      float nref = 0.f, lim = -INFINITY, sum = 0.f;     // minus the reference; how far a score may outgrow it (none yet)
      const int nc = 4 / split, c_first = grp * nc;     // 32-token chunks of a tile for this lane
      for (int j = 0; j < s.n; ++j, ++n_tile) {
        const uint32_t sbuf = tmem + TA_S + 128 * (n_tile & 1) + lanes;
        ok = ta_wait(&s_full[n_tile & 1], (n_tile >> 1) & 1, abort_v, ERR_TIMEOUT_FULL);
        if (!ok) break;
        tc05_fence_after();
        const int t0 = (s.tile0 + j) * TA_TILE;
        // The tile's weights.  Masking is fixed at compile time and done without branches: a branch per token would keep
        // the tokens' chains of multiply-add, exponential and rounding from overlapping (47 cycles a token against 6).
        auto weigh = [&](auto is_masked) {
          constexpr bool MASKED = decltype(is_masked)::value;
          bool product_over = j == 0;
#pragma unroll 1
          for (int c = c_first; c < c_first + nc; ++c) {
            uint32_t v[32];
            tmem_ld32(sbuf + 32 * c, v);
            uint32_t m = 0xffffffffu;                   // the chunk's visible tokens
            float mx = -INFINITY;
            if constexpr (MASKED) {
              const int d = t0 + 32 * c - s.len;        // drafted index of the chunk's first token
              const uint32_t behind = d <= -32 ? 0xffffffffu : (d < 0 ? (1u << (-d & 31)) - 1 : 0u);
              const uint32_t drafts = d <= -32 ? 0u : (d < 0 ? (uint32_t)(bits << (-d & 31)) : (d < 64 ? (uint32_t)(bits >> (d & 63)) : 0u));
              m = behind | drafts;
#pragma unroll
              for (int x = 0; x < 32; x += 2)
                mx = ta_max3(mx, m >> x & 1 ? __uint_as_float(v[x]) : -INFINITY, m >> (x + 1) & 1 ? __uint_as_float(v[x + 1]) : -INFINITY);
            } else {
#pragma unroll
              for (int x = 0; x < 32; x += 2) mx = ta_max3(mx, __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
            }
            const float top = mx == -INFINITY ? mx : mx * f;
            if (__any_sync(0xffffffffu, top + nref > lim)) {   // rare: the reference moves (nothing visible: it does not)
              const bool move = top + nref > lim;
              const float now = move ? Sh::BIAS - top : nref;
              const float fix = lim == -INFINITY ? 1.f : ta_exp2(now - nref);   // no weight so far: nothing to rescale
              lim = move ? Sh::GROW : lim;
              nref = now;
              sum *= fix;
              tmem_st_wait();                           // the tile's weights so far are read back below
              if (!product_over) {
                // S of this tile is there, so the product before the last has ended: one phase is open at most
                ok = ta_wait(&pv_done, (n_tile - 1) & 1, abort_v, ERR_TIMEOUT_FULL);
                if (!ok) break;
                tc05_fence_after();
                product_over = true;
              }
              if (j > 0) {
#pragma unroll 1
                for (int y = 0; y < D / 16; ++y) {
                  float o[16];
                  uint32_t w[16];
                  tmem_ld16(tmem + TA_O + lanes + 16 * y, o);
#pragma unroll
                  for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(o[x] * fix);
                  tmem_st16(tmem + TA_O + lanes + 16 * y, w);
                }
              }
#pragma unroll 1
              for (int y = c_first; y < c; ++y) {       // the tile's weights so far
                float o[16];
                uint32_t w[16];
                tmem_ld16(sbuf + 16 * y, o);
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                  const uint32_t h = __float_as_uint(o[x]);
                  float lo, hi;
                  if constexpr (RAW16) {
                    lo = __uint_as_float(h << 16);
                    hi = __uint_as_float(h & 0xffff0000u);
                  } else {
                    lo = __half2float(__ushort_as_half((unsigned short)h));
                    hi = __half2float(__ushort_as_half((unsigned short)(h >> 16)));
                  }
                  w[x] = ta_pack(lo * fix, hi * fix, RAW16);
                }
                tmem_st16(sbuf + 16 * y, w);
              }
              tmem_st_wait();
            }
            uint32_t w[16];
            float2 acc = make_float2(0.f, 0.f);
            const float2 f2 = make_float2(f, f), n2 = make_float2(nref, nref);
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float2 z = __ffma2_rn(make_float2(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1])), f2, n2);
              float2 e = make_float2(ta_exp2(z.x), ta_exp2(z.y));
              if constexpr (MASKED) {
                e.x = m >> (2 * x) & 1 ? e.x : 0.f;
                e.y = m >> (2 * x + 1) & 1 ? e.y : 0.f;
              }
              acc = __fadd2_rn(acc, e);
              w[x] = ta_pack(e.x, e.y, RAW16);
            }
            sum += acc.x + acc.y;
            tmem_st16(sbuf + 16 * c, w);                // P takes the place of S, column by column behind the reads
          }
        };
        if (t0 + TA_TILE > s.len) weigh(std::true_type{}); else weigh(std::false_type{});
        if (!ok) break;
        if (split > 1) {                                // the blocks of P off the diagonal
          const uint32_t zero[16] = {};
          const uint32_t off = sbuf + 16 * (grp ? 0 : 2);
          tmem_st16(off, zero);
          tmem_st16(off + 16, zero);
        }
        tmem_st_wait();
        tc05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[n_tile & 1]);
      }
      if (ok) ok = ta_wait(&run_done, n_seg & 1, abort_v, ERR_TIMEOUT_FULL);
      // all four warps meet before the exchange, and go on together or not at all
      const float ref = lim == -INFINITY ? -INFINITY : -nref;
      s_max[L] = ref;
      s_sum[L] = sum;
      const bool whole = ta_whole(p, s);
      const size_t slot = ta_slot(p, s);
      if (grp == 0 && real) s_out[rr] = whole ? (long long)row * p.ldo + (s.h * p.group + hg) * D : (long long)(slot * p.block + rr) * D;
      if (lane == 0) s_ok[warp] = ok;
      named_bar_sync(1, TA_SOFT * 32);
      if (!(s_ok[0] && s_ok[1] && s_ok[2] && s_ok[3])) break;
      tc05_fence_after();
      float most = -INFINITY, weight = 0.f;
      for (int g = 0; g < split; ++g) most = fmaxf(most, s_max[g * span + rr]);
      const float base = most == -INFINITY ? 0.f : most;
      for (int g = 0; g < split; ++g) weight += s_sum[g * span + rr] * ta_exp2(s_max[g * span + rr] - base);
      const float own = ta_exp2(ref - base);
      const float factor = whole ? (weight == 0.f ? 0.f : own / weight) : own;
      if (!whole && grp == 0 && rr < s.rows) {
        ta_put_stats(p, slot, rr, most, weight);
      }
      // natural element y of a chunk's columns (codes of 4 bits stand at another position inside each 8 elements)
      auto col = [](int d) { return BITS == 4 ? (d & ~7) + 2 * (d & 3) + ((d >> 2) & 1) : d; };
      if (split == 1) {
        // a lane has its row: straight from its registers
        const long long at = real ? s_out[rr] : 0;
        auto put = [&](auto is_whole) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            __syncwarp();                                // the whole warp loads; what is above and below is for lanes with a row alone
            tmem_ld32(tmem + TA_O + lanes + 32 * c, o);
            float e[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) e[x] = __uint_as_float(o[col(x)]) * factor;
            if (real) {
              if constexpr (decltype(is_whole)::value) {
#pragma unroll
                for (int x = 0; x < 32; x += 8) {
                  const uint4 w = make_uint4(ta_pack(e[x], e[x + 1], true), ta_pack(e[x + 2], e[x + 3], true),
                                             ta_pack(e[x + 4], e[x + 5], true), ta_pack(e[x + 6], e[x + 7], true));
                  *reinterpret_cast<uint4*>(p.out + at + 32 * c + x) = w;
                }
              } else {
#pragma unroll
                for (int x = 0; x < 32; x += 4)
                  *reinterpret_cast<float4*>(p.partial + at + 32 * c + x) = make_float4(e[x], e[x + 1], e[x + 2], e[x + 3]);
              }
            }
          }
        };
        if (whole) put(std::true_type{}); else put(std::false_type{});
        named_bar_sync(1, TA_SOFT * 32);
      } else {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(tmem + TA_O + lanes + 32 * c, o);
          float* dst = scratch + L * TA_PAD;
#pragma unroll
          for (int x = 0; x < 32; x += 4)
            *reinterpret_cast<float4*>(dst + x) = make_float4(__uint_as_float(o[col(x)]) * factor, __uint_as_float(o[col(x + 1)]) * factor,
                                                              __uint_as_float(o[col(x + 2)]) * factor, __uint_as_float(o[col(x + 3)]) * factor);
          named_bar_sync(1, TA_SOFT * 32);
          const int d0 = 4 * (L & 7);
          auto put = [&](auto is_whole) {
#pragma unroll 2
            for (int k = L >> 3; k < s.rows; k += 16) {
              float4 a = *reinterpret_cast<const float4*>(scratch + k * TA_PAD + d0);
              const float4 b = *reinterpret_cast<const float4*>(scratch + (64 + k) * TA_PAD + d0);
              a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
              if constexpr (decltype(is_whole)::value) {
                *reinterpret_cast<uint2*>(p.out + s_out[k] + 32 * c + d0) = make_uint2(ta_pack(a.x, a.y, true), ta_pack(a.z, a.w, true));
              } else {
                *reinterpret_cast<float4*>(p.partial + s_out[k] + 32 * c + d0) = a;
              }
            }
          };
          if (whole) put(std::true_type{}); else put(std::false_type{});
          named_bar_sync(1, TA_SOFT * 32);
        }
      }
      if (s_bad[n_seg % TA_FLAGS] && L < D) {
        // V held infinities or NaN in drafted tokens, which were left out of the products: the rows that see one get it here
        // (what they are added to was written before the last barrier)
#pragma unroll 1
        for (int k = 0; k < s.rows; ++k) {
          const int rk = s.rb * p.block + k, ik = ta_by_group(p, rk);
          const uint64_t see = ta_mask(p, s.row0 + ik, ik, s.m);
          float extra = 0.f;
#pragma unroll 1
          for (int i = 0; i < s.m; ++i) {
            const int pos = s.len + i;
            if (!(see >> i & 1) || pos < s.tile0 * TA_TILE || pos >= (s.tile0 + s.n) * TA_TILE) continue;
            const int page = ta_table(p, s.b)[pos >> p.c.page_shift];
            if ((unsigned)page >= (unsigned)p.c.n_pages) continue;
            const float val = ta_cache_value<BITS>(p.c.p.v, p.c.p.vs, p.c.p.vb,
                                                   kv_token(p.c, page, s.h, pos & ((1 << p.c.page_shift) - 1)), D, L);
            if (!isfinite(val)) extra += val;
          }
          if (extra == 0.f) continue;
          if (whole) p.out[s_out[k] + L] = __float2bfloat16_rn(__bfloat162float(p.out[s_out[k] + L]) + extra);
          else p.partial[s_out[k] + L] += extra;
        }
      }
      named_bar_sync(1, TA_SOFT * 32);
      if (L == 0) s_bad[n_seg % TA_FLAGS] = 0;
    }
  }
  tc05_fence_before();
  __syncthreads();
  if (*abort_v) {              // every copy is waited for by its reader; after a failure, those in flight get time to land
    const unsigned long long w0 = global_ns();
    while (global_ns() - w0 < 50000ull) __nanosleep(1000);
  }
  if (warp == Sh::MMA) {
    tc05_fence_after();
    tmem_dealloc(tmem, 512);
  }
  ta_end(p);
}

template <int D, int BITS, typename P>
static cudaError_t launch_wide(const P& p, cudaStream_t s) {
  using Sh = TaShape<D, BITS>;
  const cudaError_t e = cudaFuncSetAttribute(tree_attn_wide_kernel<D, BITS, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(p.grid), dim3(Sh::THREADS), Sh::SMEM, s, attr);
  return cudaLaunchKernelEx(&cfg, tree_attn_wide_kernel<D, BITS, P>, p);
}

template <typename P>
static cudaError_t launch_wide_any(const P& p, cudaStream_t s) {
  if (p.c.dim == 128)
    return p.c.bits == 16 ? launch_wide<128, 16>(p, s) : (p.c.bits == 8 ? launch_wide<128, 8>(p, s) : launch_wide<128, 4>(p, s));
  return p.c.bits == 16 ? launch_wide<64, 16>(p, s) : (p.c.bits == 8 ? launch_wide<64, 8>(p, s) : launch_wide<64, 4>(p, s));
}

cudaError_t launch_tree_attn_wide(const TreeAttnParams& p, cudaStream_t s) { return launch_wide_any(p, s); }
cudaError_t launch_tree_attn_wide(const TreeAttnOwnParams& p, cudaStream_t s) { return launch_wide_any(p, s); }

}  // namespace sv
