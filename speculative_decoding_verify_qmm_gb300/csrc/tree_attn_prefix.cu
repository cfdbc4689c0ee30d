// Attention of many rows over a shared prefix, on the 5th-generation tensor cores (PyPI page, "Prefix caching": conversations that begin
// alike share what they have in common; here a batch's rows meet those tokens once).
//
//   acc = sum_t p_t v_t,  weight = sum_t p_t,  p_t = exp(scale q . k_t - max),  t over the prefix
//
// for every row (drafted row x query head of the key head) of all the group's requests; a join adds each request's own tokens.
//
// A CTA takes two matrices of 128 rows through the same K and V tiles: S = Q K^T with Q and K in shared memory, softmax of a lane by
// one thread, P (16 bits) in S's place as the operand of O += P V.  While the softmax warps of one matrix work, the tensor cores have
// the other's products: per tile of 128 tokens 4 instructions' worth of 128 x 128 x 128, some 2048 cycles, against 128 rows x 128
// exponentials a warpgroup.  A block of up to 128 rows puts the same rows into both matrices and gives each every other tile: two
// independent sums over half of the tokens.
//
// Bound by the softmax warps where rows fill the matrices: a tile of 128 tokens takes a pair of matrices some 3500 cycles over a 16-bit cache
// (two exponentials of 32 a cycle and SM would be 1024, the products alone 2048), 1390 TFLOP/s or 0.74 of the measured rate; over codes, where
// transforming warps share the issue slots, 5600 cycles, 870 TFLOP/s.  (32 query and 8 key heads of 128: 512 rows a key head behind 16384
// tokens of an 8-bit cache 50 us.)  Few rows are bound by memory and latency: 256 rows a key head behind 8016 tokens of a 4-bit cache 30 us.
// No gain: two softmax warps a row (S is read twice as often for a maximum), an issuing warp for each matrix, scores asked for a step
// ahead, 128 scores of a row at once, five operand tiles.  Waits that spin without a time limit in the instruction cost 25 %.
//
// S, S, O and O fill the tensor memory (512 columns at 128 elements); Q is therefore read from shared memory.  The references and the
// formats of the weights are those of tree attention's tensor-core kernel.  16-bit caches come by TMA (the tail of a last tile reads as
// zeros: its page lies outside the tensor), codes through two teams of transforming warps.
#include <type_traits>

#include "tree_attn_prefix.cuh"
#include "tree_attn_tc.cuh"

namespace sv {

constexpr int PX_SOFT = 8;                         // softmax warps: 0-3 and 4-7, one lane each per row
constexpr uint32_t PX_S = 0, PX_O = 256;           // tensor-memory columns: two S (overwritten by P), two O

template <int D, int BITS>
struct PxShape {
  static constexpr int TEAMS = BITS == 16 ? 0 : 2;
  static constexpr int PROD = PX_SOFT + TEAMS * TA_TEAM, MMA = PROD + 1, THREADS = (MMA + 1) * 32;
  static constexpr int OP = TA_TILE * D * 2;
  static constexpr int QB = 128 * D * 2;           // Q of one matrix
  static constexpr int OPS = 4 * (128 / D);
  static constexpr int SMEM = 1024 + 2 * QB + OPS * OP;
  static_assert(SMEM <= 220 * 1024, "shared memory");
  static_assert(TEAMS == 0 || OPS % 2 == 0, "a team meets its slots in every turn");
  static constexpr float BIAS = BITS == 16 ? -30.f : 5.f, GROW = BITS == 16 ? -15.f : 15.f;   // as in tree attention
  static constexpr int AT_ONCE = BITS == 16 ? 64 : 32;    // a row's scores in registers at once
};

// Order of a run's operand tiles.  Two matrices on the same tiles: K0, V0, K1, V1, ...  On every other tile: K0, K1, V0, K2, V1, ...,
// V(n-2), V(n-1).
__device__ __forceinline__ bool px_item(bool pair, int e, int n, int* tile) {
  if (pair) {
    *tile = e >> 1;
    return e & 1;
  }
  if (e == 2 * n - 1) { *tile = n - 1; return true; }
  if (e < 2) { *tile = e; return false; }
  *tile = e & 1 ? (e + 1) / 2 : (e - 2) / 2;
  return !(e & 1);
}

// A run of tiles of one item in one CTA.
struct PxRun {
  int g, h, rb, rows;            // group, key head, block and its rows
  int tile0, n;                  // first tile, tiles
  int slot;                      // place of its sums
  bool pair;                     // two matrices on the same tiles
};
// The CTA's pieces are those from next to end - 1.  By key head, block, tokens.
__device__ __forceinline__ bool px_next(const PrefixParams& p, int* next, int end, PxRun* r) {
  if (*next >= end) return false;
  const int piece = *next;
  int lo = 0, hi = p.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.pieces[mid] <= piece) lo = mid; else hi = mid;
  }
  const int blocks = px_blocks(p.rows[lo]), splits = p.splits[lo], nt = px_tiles(p.tokens[lo]), i = piece - p.pieces[lo];
  const int item = i / splits, part = i - item * splits, parts = min(splits - part, end - piece);
  *next += parts;
  r->slot = p.items[lo] + item + blockIdx.x;
  r->g = lo;
  r->h = item / blocks;
  r->rb = item - r->h * blocks;
  r->pair = px_pair(p.rows[lo], r->rb);
  r->rows = min(PX_ROWS, p.rows[lo] - r->rb * PX_ROWS);
  r->tile0 = (int)((long long)part * nt / splits);
  r->n = (int)((long long)(part + parts) * nt / splits) - r->tile0;
  return true;
}

template <int D, int BITS>
__global__ void __launch_bounds__(PxShape<D, BITS>::THREADS, 1) tree_attn_prefix_kernel(const __grid_constant__ PrefixParams p) {
  using Sh = PxShape<D, BITS>;
  constexpr bool RAW16 = BITS == 16;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t op_full[Sh::OPS], op_empty[Sh::OPS];
  __shared__ uint64_t q_full[2], s_full[2], p_full[2], run_done[2], fin_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int abort_flag;
  __shared__ TaPiece pieces[RAW16 ? 1 : TA_PIECES];
  __shared__ uint64_t piece_full[TA_PIECES], piece_empty[TA_PIECES];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const ops = smem + 2 * Sh::QB;
  volatile int* abort_v = &abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::OPS; ++i) {
      mbar_init(&op_full[i], RAW16 ? 1 : TA_TEAM);
      mbar_init(&op_empty[i], 1);
    }
    for (int i = 0; i < TA_PIECES; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], TA_TEAM);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&run_done[i], 1);
    }
    mbar_init(&fin_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == Sh::MMA) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  const int all = p.pieces[p.n], first = px_first(all, p.grid, blockIdx.x), end = px_first(all, p.grid, blockIdx.x + 1);
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  pdl_trigger();               // after the wait: what comes later may then read what came before this kernel

  if (warp == Sh::PROD) {
    int u = first;
    PxRun s;
    bool ok = true;
    TaRing<RAW16 ? Sh::OPS : TA_PIECES> ring;
    const int shift = p.c.page_shift < 7 ? p.c.page_shift : 7, place_mask = (1 << p.c.page_shift) - 1;
    while (ok && px_next(p, &u, end, &s)) {
      const int32_t* const table = p.table + (size_t)p.request[s.g] * p.table_pages;
      const int tokens = p.tokens[s.g];
      constexpr int PER = D / 64;
      // this lane's tokens of a tile: a copy's (16-bit caches), or a 16-token piece
      const int my = RAW16 ? lane / PER : lane, step = RAW16 ? 1 << shift : 16, part = RAW16 ? lane - my * PER : 0;
      const bool used = my * step < TA_TILE;
      auto page_of = [&](int j) -> int {
        const int t = (s.tile0 + j) * TA_TILE + my * step;
        return j < s.n && used && t < tokens ? table[t >> p.c.page_shift] : 0;
      };
      int page_before = 0, page_k = 0, page_next = page_of(0);
      for (int i = 0; i < 2 * s.n; ++i) {
        int j;
        const bool is_v = px_item(s.pair, i, s.n, &j);
        if (!is_v) {
          page_before = page_k;
          page_k = page_next;
          page_next = page_of(j + 1);
        }
        int page = is_v && !s.pair && i != 2 * s.n - 1 ? page_before : page_k;
        ok = ta_wait(RAW16 ? &op_empty[ring.slot] : &piece_empty[ring.slot], ring.phase ^ 1, abort_v, ERR_TIMEOUT_EMPTY);
        if (!ok) break;
        const int t0 = (s.tile0 + j) * TA_TILE, t = t0 + my * step;
        if ((unsigned)page >= (unsigned)p.c.n_pages) {
          raise_error(ERR_BAD_INPUT);
          page = 0;                                    // stay inside the arrays: the result is undefined
        }
        if constexpr (RAW16) {
          if (lane == 0) mbar_arrive_expect_tx(&op_full[ring.slot], Sh::OP);
          __syncwarp();
          if (used) {
            // past the end a slab that is not there: zeros
            const int slab = t < tokens ? page * p.c.heads + s.h : p.c.n_pages * p.c.heads;
            uint8_t* dst = ops + ring.slot * Sh::OP + part * (TA_TILE * 128) + (my << shift) * 128;
            tma_load_3d_plain(dst, is_v ? &p.tv : &p.tk, &op_full[ring.slot], part * 64, t < tokens ? t & place_mask : 0, slab);
          }
        } else {
          TaPiece& x = pieces[ring.slot];
          if (used) {
            const size_t tok = t < tokens ? kv_token(p.c, page, s.h, t & place_mask) : 0;
            x.codes[lane] = (is_v ? p.c.p.v : p.c.p.k) + tok * (D * BITS / 8);
            x.scales[lane] = (is_v ? p.c.p.vs : p.c.p.ks) + tok * (D / GROUP);
            x.biases[lane] = (is_v ? p.c.p.vb : p.c.p.kb) + tok * (D / GROUP);
          }
          if (lane == 8) {
            x.valid = x.drafted = tokens - t0;
            x.is_v = is_v;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&piece_full[ring.slot]);
        }
        ring.next();
      }
    }
    if constexpr (!RAW16) {                            // the end: one descriptor for each team
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
    TaRing<Sh::OPS> ring;
    uint32_t n_q[2] = {0, 0}, n_p[2] = {0, 0};          // phases seen
    bool ok = true;
    constexpr uint32_t ID_S = f16_idesc_ex(128, TA_TILE, RAW16, false), ID_O = f16_idesc_ex(128, D, RAW16, true);
    const bool issuer = elect_one();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t q0 = (__shfl_sync(0xffffffffu, smem_u32(smem), 0) & 0x3FFFFu) >> 4, ops0 = q0 + (2 * Sh::QB >> 4);
    constexpr uint32_t HI = (1024u >> 4) | (1u << 14) | (2u << 29);
    constexpr uint32_t LO_K = 1u << 16, LO_V = (uint32_t)(TA_TILE * 128 >> 4) << 16;
    auto desc = [](uint32_t lo) { return (uint64_t)HI << 32 | lo; };
    auto scores = [&](int x, uint32_t base) {           // S of matrix x
      if (issuer) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t at = (kk >> 2) * (128 * 128 >> 4) + (kk & 3) * 2;
          tc05_mma_f16(tm + PX_S + 128 * x, desc((q0 + x * (Sh::QB >> 4) + at) | LO_K), desc((base + at) | LO_K), ID_S, kk > 0);
        }
        tc05_commit(&s_full[x]);
      }
    };
    auto values = [&](int x, uint32_t base, bool first, bool last) {   // O of matrix x
      if (issuer) {
#pragma unroll
        for (int kk = 0; kk < TA_TILE / 16; ++kk)
          tc05_mma_f16_ts(tm + PX_O + D * x, tm + PX_S + 128 * x + 8 * kk, (base + kk * (2048 >> 4)) | LO_V, HI, ID_O, !first || kk > 0);
        if (last) tc05_commit(&run_done[x]);
      }
    };
    auto full = [&](uint32_t* base) -> bool {           // the next operand tile
      if (!ta_wait(&op_full[ring.slot], ring.phase, abort_v, ERR_TIMEOUT_FULL)) return false;
      tc05_fence_after();
      *base = ops0 + ring.slot * (Sh::OP >> 4);
      return true;
    };
    auto weights = [&](int x) -> bool {
      const bool got = ta_wait(&p_full[x], n_p[x]++ & 1, abort_v, ERR_TIMEOUT_FULL);
      tc05_fence_after();
      return got;
    };
    auto query = [&](int x) -> bool {
      const bool got = ta_wait(&q_full[x], n_q[x]++ & 1, abort_v, ERR_TIMEOUT_FULL);
      tc05_fence_after();
      return got;
    };
    int u = first;
    PxRun s;
    while (ok && px_next(p, &u, end, &s)) {
      const int n = __shfl_sync(0xffffffffu, s.n, 0);
      uint32_t kb = 0, vb = 0;
      if (s.pair) {
        for (int i = 0; i <= n && ok; ++i) {
          int slot_v = 0, slot_k = 0;
          if (i > 0) {
            ok = full(&vb);
            slot_v = ring.slot;
            ring.next();
          }
          for (int x = 0; x < 2 && ok; ++x) {
            if (i > 0) {
              ok = weights(x);
              if (!ok) break;
              values(x, vb, i == 1, i == n);
              if (x == 1 && issuer) tc05_commit(&op_empty[slot_v]);
            }
            if (i < n) {
              if (x == 0) {
                ok = full(&kb);
                slot_k = ring.slot;
                ring.next();
              }
              if (ok && i == 0) ok = query(x);
              if (!ok) break;
              scores(x, kb);
              if (x == 1 && issuer) tc05_commit(&op_empty[slot_k]);
            }
            __syncwarp();
          }
        }
      } else {
        for (int e = 0; e < n + 2 && ok; ++e) {
          const int x = e & 1;
          if (e >= 2) {
            ok = full(&vb) && weights(x);
            if (!ok) break;
            values(x, vb, e < 4, e >= n);
            if (issuer) tc05_commit(&op_empty[ring.slot]);
            ring.next();
          }
          if (e < n) {
            ok = full(&kb);
            if (ok && e < 2) ok = query(x);
            if (!ok) break;
            scores(x, kb);
            if (issuer) tc05_commit(&op_empty[ring.slot]);
            ring.next();
          }
          __syncwarp();
        }
      }
    }
    // no MMA may still be running when the tensor memory is freed: this wait ignores the abort flag and ends only on completion or the
    // time limit
    if (issuer) {
      tc05_commit(&fin_bar);
      volatile int never = 0;
      mbar_wait_bounded(&fin_bar, 0, &never);
    }
    __syncwarp();
  } else if (warp >= PX_SOFT) {
    if constexpr (!RAW16)
      ta_transform<D, BITS, Sh::TEAMS, Sh::OPS, false>(ops, op_full, op_empty, pieces, piece_full, piece_empty, nullptr, abort_v,
                                                       (warp - PX_SOFT) / TA_TEAM, (warp - PX_SOFT) % TA_TEAM, lane);
  } else {
    // ============================================================ softmax, and the ends of runs
    const int x = warp >> 2, L = threadIdx.x & 127;     // matrix, and its lane
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t sbuf = tmem + PX_S + 128 * x + lanes, obuf = tmem + PX_O + D * x + lanes;
    uint8_t* const qbuf = smem + x * Sh::QB + L * 128;
    uint32_t n_s = 0, n_run = 0;                        // phases of s_full, run_done
    bool ok = true;
    int u = first;
    PxRun s;
    while (ok && px_next(p, &u, end, &s)) {
      const int rr = s.pair ? 128 * x + L : L;          // row of the block
      const bool real = rr < s.rows;
      const int r = s.rb * PX_ROWS + rr;
      const int di = real ? r / p.heads_per : 0, hg = real ? r - di * p.heads_per : 0;
      const int n = s.pair ? s.n : (s.n + 1 - x) >> 1;  // this matrix's tiles
      float f = 0.f;                                    // score -> exponent of 2
      if (n) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (size_t)(p.row0[s.g] + di) * p.ldq + (s.h * p.heads_per + hg) * D);
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
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = real ? src[c] : make_uint4(0, 0, 0, 0);
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if constexpr (RAW16) {
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] ^= minus ? 0x80008000u : 0u;
          } else {
            float e[8];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              e[2 * y] = __uint_as_float(w[y] << 16) * up;
              e[2 * y + 1] = __uint_as_float(w[y] & 0xffff0000u) * up;
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = BITS == 4 ? ta_pack(e[y], e[y + 4], false) : ta_pack(e[2 * y], e[2 * y + 1], false);
          }
          *reinterpret_cast<uint4*>(qbuf + (c >> 3) * (128 * 128) + (((c & 7) ^ (L & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        tc05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[x]);
      }
      float nref = 0.f, lim = -INFINITY, sum = 0.f;     // minus the reference; how far a score may outgrow it (none yet)
      const int tokens = p.tokens[s.g];
      for (int i = 0; i < n; ++i, ++n_s) {
        ok = ta_wait(&s_full[x], n_s & 1, abort_v, ERR_TIMEOUT_FULL);   // and with it the product before: they end in order
        if (!ok) break;
        tc05_fence_after();
        const int j = s.pair ? i : 2 * i + x, left = tokens - (s.tile0 + j) * TA_TILE;
        auto weigh = [&](auto is_masked) {
          constexpr bool MASKED = decltype(is_masked)::value;
          constexpr int NB = Sh::AT_ONCE;                 // columns at once
#pragma unroll
          for (int c0 = 0; c0 < TA_TILE; c0 += NB) {
            uint32_t v[NB];
#pragma unroll
            for (int c = 0; c < NB; c += 32) tmem_ld32_async(sbuf + c0 + c, v + c);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < NB; c += 32) tmem_arrived(v + c);
            if constexpr (MASKED) {
#pragma unroll
              for (int y = 0; y < NB; ++y) v[y] = c0 + y < left ? v[y] : 0xff800000u;   // -inf
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int y = 0; y < NB; y += 8)
#pragma unroll
              for (int z = 0; z < 4; ++z) m4[z] = ta_max3(m4[z], __uint_as_float(v[y + 2 * z]), __uint_as_float(v[y + 2 * z + 1]));
            const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            const float top = mx == -INFINITY ? mx : mx * f;
            if (__any_sync(0xffffffffu, top + nref > lim)) {   // rare: the reference moves (nothing visible: it does not)
              const bool move = top + nref > lim;
              const float now = move ? Sh::BIAS - top : nref;
              const float fix = lim == -INFINITY ? 1.f : ta_exp2(now - nref);   // no weight so far: nothing to rescale
              lim = move ? Sh::GROW : lim;
              nref = now;
              sum *= fix;
              if (i > 0) {
#pragma unroll 1
                for (int y = 0; y < D / 16; ++y) {
                  float o[16];
                  uint32_t w[16];
                  tmem_ld16(obuf + 16 * y, o);
#pragma unroll
                  for (int z = 0; z < 16; ++z) w[z] = __float_as_uint(o[z] * fix);
                  tmem_st16(obuf + 16 * y, w);
                }
              }
              if (c0 > 0) tmem_st_wait();               // the tile's weights so far are read back
#pragma unroll 1
              for (int y = 0; y < c0 / 32; ++y) {
                float o[16];
                uint32_t w[16];
                tmem_ld16(sbuf + 16 * y, o);
#pragma unroll
                for (int z = 0; z < 16; ++z) {
                  const uint32_t h = __float_as_uint(o[z]);
                  float lo, hi;
                  if constexpr (RAW16) {
                    lo = __uint_as_float(h << 16);
                    hi = __uint_as_float(h & 0xffff0000u);
                  } else {
                    lo = __half2float(__ushort_as_half((unsigned short)h));
                    hi = __half2float(__ushort_as_half((unsigned short)(h >> 16)));
                  }
                  w[z] = ta_pack(lo * fix, hi * fix, RAW16);
                }
                tmem_st16(sbuf + 16 * y, w);
              }
            }
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 f2 = make_float2(f, f), n2 = make_float2(nref, nref);
#pragma unroll
            for (int c = 0; c < NB; c += 32) {
              uint32_t w[16];
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                const float2 z = __ffma2_rn(make_float2(__uint_as_float(v[c + 2 * y]), __uint_as_float(v[c + 2 * y + 1])), f2, n2);
                float2 e = make_float2(ta_exp2(z.x), ta_exp2(z.y));
                if constexpr (MASKED) {                   // (a factor of zero makes NaN of -inf)
                  e.x = c0 + c + 2 * y < left ? e.x : 0.f;
                  e.y = c0 + c + 2 * y + 1 < left ? e.y : 0.f;
                }
                acc[y & 1] = __fadd2_rn(acc[y & 1], e);
                w[y] = ta_pack(e.x, e.y, RAW16);
              }
              tmem_st16(sbuf + (c0 + c) / 2, w);          // P takes the place of S, behind the reads
            }
            sum += (acc[0].x + acc[1].x) + (acc[0].y + acc[1].y);
          }
        };
        if (left < TA_TILE) weigh(std::true_type{}); else weigh(std::false_type{});
        tmem_st_wait();
        tc05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      if (n) {
        ok = ta_wait(&run_done[x], n_run++ & 1, abort_v, ERR_TIMEOUT_FULL);
        if (!ok) break;
        tc05_fence_after();
      }
      const size_t at = (size_t)s.slot * PX_ROWS + 128 * x + L;
      if (real) {
        ta_put_sector(p.stats + at * TA_STAT, lim == -INFINITY ? -INFINITY : -nref, sum);
      }
      if (n) {
        // natural element y of a chunk's columns (codes of 4 bits stand at another position inside each 8 elements)
        auto col = [](int d) { return BITS == 4 ? (d & ~7) + 2 * (d & 3) + ((d >> 2) & 1) : d; };
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          __syncwarp();                                  // the whole warp loads; what is above and below is for lanes with a row alone
          tmem_ld32(obuf + 32 * c, o);
          if (real) {
#pragma unroll
            for (int y = 0; y < 32; y += 8) {            // a lane has a row: whole sectors
              uint32_t v[8];
#pragma unroll
              for (int z = 0; z < 8; ++z) v[z] = o[col(y + z)];
              ta_store8(p.partial + at * D + 32 * c + y, v);
            }
          }
        }
      }
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
}

template <int D, int BITS>
static cudaError_t launch_prefix(const PrefixParams& p, cudaStream_t s) {
  using Sh = PxShape<D, BITS>;
  const cudaError_t e = cudaFuncSetAttribute(tree_attn_prefix_kernel<D, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(p.grid), dim3(Sh::THREADS), Sh::SMEM, s, attr);
  return cudaLaunchKernelEx(&cfg, tree_attn_prefix_kernel<D, BITS>, p);
}

cudaError_t launch_tree_attn_prefix(const PrefixParams& p, cudaStream_t s) {
  if (p.c.dim == 128)
    return p.c.bits == 16 ? launch_prefix<128, 16>(p, s) : (p.c.bits == 8 ? launch_prefix<128, 8>(p, s) : launch_prefix<128, 4>(p, s));
  return p.c.bits == 16 ? launch_prefix<64, 16>(p, s) : (p.c.bits == 8 ? launch_prefix<64, 8>(p, s) : launch_prefix<64, 4>(p, s));
}

}  // namespace sv
