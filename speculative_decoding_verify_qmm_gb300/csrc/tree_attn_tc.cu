// Attention of the drafted rows over the paged cache, on the 5th-generation tensor cores (mlx-dspark wiki page,
// "Architecture": the target verifies the drafted block in one forward over its cache).
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - max)
//
// The drafted rows of a request times the query heads of one key head are the N columns of the products (16 .. 128; more
// rows are several items), and the cached tokens and the head's elements are their 128 lanes, so a product costs what its
// rows need:
//   S  [token x row] = K Q^T       K from shared memory (A operand, K-major), Q resident there (B operand)
//   O  [elem x row] += V^T P^T     V as it lies ([token][elem], MN-major A), P [token][row] in shared memory (MN-major B)
//   L  [any x row]  += 1 P^T       the rows' weights, from a tile of ones
// S, O and L are in tensor memory.  A thread owns one token of the tile, so its softmax needs no neighbour: the weight is
// 2^(S f_r - ref_r) with a reference per row that all threads share.  The reference moves only when some score has outgrown
// it (by 2^15 in fp16, 2^60 in bf16): one barrier with an OR per tile finds that out,
// after P is written; then, rarely, the tile's row maxima are taken, O and L are rescaled, and P is written again.
// The end of an item needs no exchange: a lane has one element of every row.
//
// Bound by memory for few rows; tiles of 128 tokens, dealt to one CTA per SM.  16-bit caches go from TMA to the tensor cores
// untouched.  Codes are dequantized by three teams of four warps into fp16 in the operand layout, fp16(s * c + b) with the
// exact code (half an fp16 step), and Q enters as fp16 scaled by a power of two per row, exact for every bf16 value
// within 2^29 of the row's largest.
#include <type_traits>

#include "sv_tc05.cuh"
#include "tree_attn.cuh"

namespace sv {

constexpr int TA_TILE = 128;                       // tokens per tile: the lanes of tensor memory
constexpr int TA_GROUP = 4, TA_SOFT = 2 * TA_GROUP;  // two groups of four softmax warps (0-7), for even and odd tiles
constexpr int TA_TEAM = 4;                         // warps of a transforming team
constexpr int TA_FLAGS = 16;                       // segments whose flags are alive at once (ring depth / 2 at most)
constexpr uint32_t TA_S = 0, TA_O = 256, TA_L = 384;  // tensor-memory columns: the S buffers; O; L

// NB: rows per item at most.  Warps: softmax, transforming teams, the copying warp, the MMA warp.
template <int D, int BITS, int NB>
struct TaShape {
  // Items of up to 64 rows: two issuing warps, one for each product (an instruction takes its warp some 70 cycles to issue,
  // more than such an item's products run), and a ring in which K and V alternate.  Wider items need the shared memory for
  // Q and P: three slots, one issuing warp, K a tile ahead of V.
  static constexpr bool SPLIT = NB == 64;
  static constexpr int SB = 256 / NB;                                              // S buffers
  static constexpr int TEAMS = BITS == 16 ? 1 : (SPLIT ? 4 : 3);
  static constexpr int PROD = TA_SOFT + TEAMS * TA_TEAM, MMA = PROD + 1, MMA2 = MMA + SPLIT, THREADS = (MMA2 + 1) * 32;
  static constexpr int OP = TA_TILE * D * 2;                                       // one operand tile, 16 bits a value
  static constexpr int Q = NB * D * 2, P = NB / 64 * TA_TILE * 128, ONES = 1024;
  static constexpr int FIT = (218 * 1024 - Q - 2 * P - ONES) / OP;
  static constexpr int OPS = BITS == 16 ? (FIT > 10 ? 10 : (SPLIT ? FIT & ~1 : FIT)) : (SPLIT ? 4 : 3);  // ring of operand tiles
  static constexpr int SMEM = 1024 + OPS * OP + Q + 2 * P + ONES;
  // A weight enters the second product in 16 bits: bf16 has room for any score difference that fp32 sums can bear, fp16
  // for 2^15; there the reference starts 2^5 below the largest score of its tile, so that weights down to 2^-29 of it keep
  // all their bits.
  static constexpr float BIAS = BITS == 16 ? 0.f : 5.f, GROW = BITS == 16 ? 60.f : 15.f;
  static_assert(SMEM <= 220 * 1024, "shared memory");
  static_assert(OPS % TEAMS == 0, "a team meets its slots in every turn, so it sees every phase of their barriers");
  static_assert(!SPLIT || OPS % 2 == 0, "each product's slots are its own");
  static_assert(OPS <= 2 * TA_FLAGS - 4, "flags");
};

// Order of a run's operand tiles.  SPLIT: K0, V0, K1, V1, ...; else K0, K1, V0, K2, V1, ..., V(n-1).  Sets the tile; true: V.
template <bool SPLIT>
__device__ __forceinline__ bool ta_item(int e, int n, int* tile) {
  if constexpr (SPLIT) {
    *tile = e >> 1;
    return e & 1;
  }
  const bool is_v = e == 2 * n - 1 || (e > 0 && !(e & 1));
  *tile = e == 2 * n - 1 ? n - 1 : (is_v ? e / 2 - 1 : (e + 1) / 2);
  return is_v;
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

// One 32-bit word of codes as fp16 pairs s * c + b (two fp16 steps: an exact subtraction of 1024, one fused
// multiply-add).  8-bit: pairs (c0, c1), (c2, c3).  4-bit: pairs (c_j, c_j+4): inside each 8 elements position q holds
// element q / 2 + 4 (q % 2), an order that Q is laid out in too and that the output undoes.
template <int BITS>
__device__ __forceinline__ void ta_dequant(uint32_t w, __half2 s2, __half2 b2, uint32_t* out) {
  const __half2 k1024 = __half2half2(__ushort_as_half((unsigned short)0x6400));
  if constexpr (BITS == 8) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t biased = __byte_perm(w, 0x64646464u, j ? 0x4342 : 0x4140);
      const __half2 v = __hfma2(s2, __hsub2(*reinterpret_cast<const __half2*>(&biased), k1024), b2);
      out[j] = *reinterpret_cast<const uint32_t*>(&v);
    }
  } else {
    const __half2 k16 = __half2half2(__ushort_as_half((unsigned short)0x2c00)), k64 = __half2half2(__ushort_as_half((unsigned short)0xd400));
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // a nibble four bits up reads as 1024 + 16 c: one multiply-add (exact) instead of a shift
      const uint32_t x = j < 2 ? w : w >> 8;
      const uint32_t biased = (x & (j & 1 ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;
      const __half2 h = *reinterpret_cast<const __half2*>(&biased);
      const __half2 v = __hfma2(s2, j & 1 ? __hfma2(h, k16, k64) : __hsub2(h, k1024), b2);
      out[j] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// 16 bytes that are read once: kept out of L1.
__device__ __forceinline__ uint4 ld_stream16(const uint8_t* a) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(a));
  return v;
}

// max of three (NaN operands are passed over, as by fmaxf)
__device__ __forceinline__ float ta_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A position in a ring of N slots and the parity of its current turn.
template <int N>
struct TaRing {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int by = 1) {   // by <= N
    slot += by;
    if (slot >= N) {
      slot -= N;
      phase ^= 1;
    }
  }
};

// A wait that leaves its issue slots to the others: the hardware suspends the thread for up to the hinted time.
__device__ __forceinline__ bool ta_poll(uint64_t* bar, uint32_t parity, volatile int* abort_v) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(100000u)
      : "memory");
  return ok || mbar_wait_bounded(bar, parity, abort_v);
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

// Barrier of the softmax warps that returns whether any of them brought true.
template <int THREADS>
__device__ __forceinline__ bool ta_any(int id, bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)mine), "r"(id), "n"(THREADS)
      : "memory");
  return r != 0;
}
// Order-preserving key of an fp32 value as a signed integer, and back.
__device__ __forceinline__ int ta_key(float f) {
  const int b = __float_as_int(f);
  return b >= 0 ? b : b ^ 0x7fffffff;
}
__device__ __forceinline__ float ta_unkey(int k) { return __int_as_float(k >= 0 ? k : k ^ 0x7fffffff); }

template <int D, int BITS, int NB>
__global__ void __launch_bounds__(TaShape<D, BITS, NB>::THREADS, 1) tree_attn_kernel(const __grid_constant__ TreeAttnParams p) {
  using Sh = TaShape<D, BITS, NB>;
  constexpr bool RAW16 = BITS == 16;
  extern __shared__ uint8_t smem_raw[];
  // operand slots: copied into (16-bit caches only), ready for the tensor cores, read
  __shared__ uint64_t load_full[Sh::OPS], op_full[Sh::OPS], op_empty[Sh::OPS];
  __shared__ uint64_t q_full, s_full[Sh::SB], s_free[Sh::SB], run_done, fin_bar[2];
  __shared__ uint64_t p_full[2], pv_done[2], checked[2];  // [tile parity]
  __shared__ uint32_t s_tmem;
  __shared__ int abort_flag, s_bad[TA_FLAGS];
  __shared__ TaPlan plan;
  __shared__ TaPiece pieces[RAW16 ? 1 : TA_PIECES];     // caches of codes: filled by the copying warp, read by one team each
  __shared__ uint64_t piece_full[TA_PIECES], piece_empty[TA_PIECES];
  // per row of the block: score factor and minus the reference (two rows together), mask, where the row is written
  __shared__ float4 s_fr[NB / 2];
  __shared__ uint64_t s_mask[NB];
  __shared__ long long s_out[NB];
  // of a slow tile: row maxima per warp, rescaling factors, whether some row has no reference yet
  __shared__ int s_key[TA_GROUP][NB];
  __shared__ float s_fix[NB];
  __shared__ bool s_unset[NB];                           // rows without a reference yet
  __shared__ int s_failed[TA_SOFT];
  __shared__ volatile int s_version, s_all_set;          // of the references: counts their changes; every row has one
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const ops = smem;
  uint8_t* const s_q = smem + Sh::OPS * Sh::OP;
  uint8_t* const s_p = s_q + Sh::Q;
  uint8_t* const s_ones = s_p + 2 * Sh::P;
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
    mbar_init(&q_full, 1);
    for (int i = 0; i < Sh::SB; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&p_full[i], 1);
      mbar_init(&pv_done[i], 1);
      mbar_init(&checked[i], 1);
    }
    mbar_init(&run_done, 1);
    mbar_init(&fin_bar[0], 1);
    mbar_init(&fin_bar[1], 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < TA_FLAGS) s_bad[threadIdx.x] = 0;
  if (threadIdx.x == 0) s_version = 0;
  if (threadIdx.x >= 64 && threadIdx.x < 128) {          // 1 KB of ones, in the operand type
    const uint32_t one = RAW16 ? 0x3f803f80u : 0x3c003c00u;
    reinterpret_cast<uint4*>(s_ones)[threadIdx.x - 64] = make_uint4(one, one, one, one);
    fence_proxy_async_smem();
  }
  if (warp == Sh::MMA) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();             // after the wait: the join may then read what this kernel's predecessors wrote before its own
  if (warp == 0) ta_plan(p, &plan, blockIdx.x == 0);
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
      TaSeg s;
      for (long long u = u0; ok && ta_next(p, plan, &u, u0, u1, &s);) {
        // the table's entry for this lane's chunk of tile j, checked when it is used: the load is a tile ahead
        auto page_of = [&](int j) -> int {
          const int t = (s.tile0 + j) * TA_TILE + (my_chunk << shift);
          if (j >= s.n || my_chunk >= (TA_TILE >> shift) || t >= s.total) return 0;
          return p.table[(size_t)s.b * p.table_pages + (t >> p.c.page_shift)];
        };
        int page_before = 0, page_k = 0, page_next = page_of(0);   // of the last two K tiles, and the next one's
        for (int i = 0; i < 2 * s.n; ++i) {
          int j;
          const bool is_v = ta_item<Sh::SPLIT>(i, s.n, &j);
          if (!is_v) {
            page_before = page_k;
            page_k = page_next;
            page_next = page_of(j + 1);
          }
          int page = !Sh::SPLIT && is_v && i != 2 * s.n - 1 ? page_before : page_k;
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
      TaSeg s;
      for (long long u = u0; ok && ta_next(p, plan, &u, u0, u1, &s); ++n_seg) {
        auto page_of = [&](int j) -> int {             // of 16-token piece `lane` of tile j; checked when it is used
          const int t = (s.tile0 + j) * TA_TILE + 16 * lane;
          if (j >= s.n || lane >= TA_TILE / 16 || t >= s.total) return 0;
          return p.table[(size_t)s.b * p.table_pages + (t >> p.c.page_shift)];
        };
        int page_before = 0, page_k = 0, page_next = page_of(0);   // of the last two K tiles, and the next one's
        for (int i = 0; i < 2 * s.n; ++i) {
          int j;
          const bool is_v = ta_item<Sh::SPLIT>(i, s.n, &j);
          if (!is_v) {
            page_before = page_k;
            page_k = page_next;
            page_next = page_of(j + 1);
          }
          int page = !Sh::SPLIT && is_v && i != 2 * s.n - 1 ? page_before : page_k;
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
  } else if (warp >= Sh::MMA) {
    // ============================================================ MMA issue
    // The whole warp runs the loop and one lane issues, so that descriptors and addresses live in uniform registers.
    {
      TaRing<Sh::OPS> ring;
      if (Sh::SPLIT && warp == Sh::MMA2) ring.next();   // V's slots are the odd ones
      uint32_t n_q = 0, n_s = 0, n_p = 0;               // phases seen of each barrier
      bool ok = true;
      const bool issuer = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      auto start = [&](const uint8_t* at) { return (__shfl_sync(0xffffffffu, smem_u32(at), 0) & 0x3FFFFu) >> 4; };
      const uint32_t ops0 = start(ops), q0 = start(s_q), p0 = start(s_p), ones0 = start(s_ones);
      // Descriptors differ in the start address and the leading byte offset (bits 16-29 of the low word; unused by K-major
      // operands).  A head of 64 elements fills 64 of V's lanes; the upper 64 read the same block again.
      constexpr uint32_t HI = (1024u >> 4) | (1u << 14) | (2u << 29), HI_ONES = (1u << 14) | (2u << 29);
      constexpr uint32_t LO_K = 1u << 16, LO_V = (D == 128 ? (uint32_t)(TA_TILE * 128 >> 4) : 0u) << 16,
                         LO_P = (uint32_t)(TA_TILE * 128 >> 4) << 16;
      TaSeg s;
      for (long long u = u0; ok && ta_next(p, plan, &u, u0, u1, &s);) {
        int n, rows;
        {
          n = __shfl_sync(0xffffffffu, s.n, 0);
          rows = __shfl_sync(0xffffffffu, s.rows, 0);
        }
        const int N = (rows + 15) & ~15;
        const uint32_t id_s = f16_idesc_ex(TA_TILE, N, RAW16, false, false), id_o = f16_idesc_ex(TA_TILE, N, RAW16, true, true),
                       id_l = f16_idesc_ex(TA_TILE, N, RAW16, false, true);
        // S = K Q^T of tile n_s
        auto scores = [&](uint32_t base) {
          const uint32_t d = tm + TA_S + NB * (n_s % Sh::SB), lo = base | LO_K, qlo = q0 | LO_K;
          if (issuer) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc05_mma_f16_lohi(d, lo + (kk >> 2) * (TA_TILE * 128 >> 4) + (kk & 3) * 2, HI,
                                qlo + (kk >> 2) * (NB * 128 >> 4) + (kk & 3) * 2, HI, id_s, kk > 0);
            tc05_commit(&s_full[n_s % Sh::SB]);
            tc05_commit(&op_empty[ring.slot]);
          }
          ++n_s;
        };
        // O += V^T P^T and L += 1 P^T of tile n_p
        auto values = [&](uint32_t base, bool first, bool last) {
          const uint32_t lo = base | LO_V, plo = (p0 + (n_p & 1) * (Sh::P >> 4)) | LO_P, ones = ones0 | LO_K;
          if (issuer) {
#pragma unroll
            for (int kk = 0; kk < TA_TILE / 16; ++kk) {
              tc05_mma_f16_lohi(tm + TA_O, lo + kk * (2048 >> 4), HI, plo + kk * (2048 >> 4), HI, id_o, !first || kk > 0);
              tc05_mma_f16_lohi(tm + TA_L, ones, HI_ONES, plo + kk * (2048 >> 4), HI, id_l, !first || kk > 0);
            }
            tc05_commit(&pv_done[n_p & 1]);
            tc05_commit(&op_empty[ring.slot]);
            if (last) tc05_commit(&run_done);
          }
          ++n_p;
        };
        if constexpr (Sh::SPLIT) {
          if (warp == Sh::MMA) {
            ok = ta_wait(&q_full, n_q++ & 1, abort_v, ERR_TIMEOUT_FULL);
            for (int j = 0; j < n && ok; ++j) {
              if (n_s >= Sh::SB) ok = ta_wait(&s_free[n_s % Sh::SB], (n_s / Sh::SB - 1) & 1, abort_v, ERR_TIMEOUT_FULL);
              if (ok) ok = ta_wait(&op_full[ring.slot], ring.phase, abort_v, ERR_TIMEOUT_FULL);
              if (!ok) break;
              tc05_fence_after();
              scores(ops0 + ring.slot * (Sh::OP >> 4));
              __syncwarp();
              ring.next(2);
            }
          } else {
            for (int j = 0; j < n && ok; ++j) {
              ok = ta_wait(&op_full[ring.slot], ring.phase, abort_v, ERR_TIMEOUT_FULL);
              if (ok) ok = ta_wait(&p_full[n_p & 1], (n_p >> 1) & 1, abort_v, ERR_TIMEOUT_FULL);
              if (!ok) break;
              tc05_fence_after();
              values(ops0 + ring.slot * (Sh::OP >> 4), j == 0, j == n - 1);
              __syncwarp();
              ring.next(2);
            }
          }
        } else {
          ok = ta_wait(&q_full, n_q++ & 1, abort_v, ERR_TIMEOUT_FULL);
          for (int i = 0; i < 2 * n && ok; ++i) {
            int j;
            const bool is_v = ta_item<false>(i, n, &j);
            ok = ta_wait(&op_full[ring.slot], ring.phase, abort_v, ERR_TIMEOUT_FULL);
            if (ok && is_v) ok = ta_wait(&p_full[n_p & 1], (n_p >> 1) & 1, abort_v, ERR_TIMEOUT_FULL);
            if (ok && !is_v && n_s >= Sh::SB) ok = ta_wait(&s_free[n_s % Sh::SB], (n_s / Sh::SB - 1) & 1, abort_v, ERR_TIMEOUT_FULL);
            if (!ok) break;
            tc05_fence_after();
            if (is_v) values(ops0 + ring.slot * (Sh::OP >> 4), j == 0, j == n - 1);
            else scores(ops0 + ring.slot * (Sh::OP >> 4));
            __syncwarp();
            ring.next();
          }
        }
      }
      // no MMA may still be running when the tensor memory is freed: this wait
      // ignores the abort flag and ends only on completion or the time limit
      if (issuer) {
        uint64_t* const mine = &fin_bar[warp - Sh::MMA];
        tc05_commit(mine);
        volatile int never = 0;
        mbar_wait_bounded(mine, 0, &never);
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
      TaSeg s;
      for (long long u = u0; ok && ta_next(p, plan, &u, u0, u1, &s); ++n_seg) {
        for (int i = 0; i < 2 * s.n; ++i, ring.next()) {
          int j;
          const bool is_v = ta_item<Sh::SPLIT>(i, s.n, &j);
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
      // Where this lane's chunks go in its first row; the rows of later steps differ in the swizzle by one bit at most.
      uint32_t to[NCH];
#pragma unroll
      for (int y = 0; y < NCH; ++y)
        to[y] = smem_u32(ops) + (part * PERT / 64) * (TA_TILE * 128) + (32 * tw + sub) * 128 + (((c0 + (y ^ sel)) ^ (sub & 7)) << 4);
      TaRing<Sh::OPS> ring;
      TaRing<TA_PIECES> ahead, here;
      ring.next(team);
      ahead.next(team);
      here.next(team);
      uint4 raw[LPT];
      uint32_t sc = 0, bi = 0;                          // scales and biases of this lane's token (two groups, or one)
      const uint8_t* at[2] = {};                        // the warp's two 16-token halves
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
          // (past the end, the cache's first tokens stand in: the loads need no branch, and nothing comes of them)
          at[hf] = (is_v ? p.c.p.v : p.c.p.k) + (tok < 0 ? 0 : tok) * ROWB + lane * 16;
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
        ahead.next(Sh::TEAMS);
        return true;
      };
      auto fetch = [&](int i) {
        const int hf = i * TPS / 16;
        raw[i] = ld_stream16(at[hf] + (i * TPS - 16 * hf) * ROWB);
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
        const uint32_t dst = ring.slot * Sh::OP;
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
#pragma unroll
          for (int y = 0; y < NCH; ++y)
            sts128((to[y] ^ (((i * TPS) & 7) << 4)) + dst + i * TPS * 128, o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
        }
        fence_proxy_async_smem();  // the tensor cores read these writes through the async proxy
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&op_full[ring.slot]);
          mbar_arrive(&piece_empty[here.slot]);
        }
        ring.next(Sh::TEAMS);
        here.next(Sh::TEAMS);
        ok = locate();
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < LPT; ++i) fetch(i);
      }
    }
  } else {
    // ============================================================ softmax, and the ends of segments
    // The groups take turns: one weighs its tile while the other's is in the second product.  References change rarely and
    // one tile at a time: a tile is "checked" once it is known that its scores fit them (or they have been changed to), and
    // the next tile is not before.  A group that weighed its tile with references that changed meanwhile weighs it again.
    const int group = warp / TA_GROUP, gw = warp % TA_GROUP, bar = 1 + group;
    const int t = threadIdx.x % 128;                    // this thread's token of a tile, and lane of tensor memory
    const uint32_t lanes = (uint32_t)(32 * gw) << 16;
    uint32_t n0 = 0;                                    // tiles of the runs before: a tile's number gives group and phases
    int n_seg = 0;
    TaSeg s;
    for (long long u = u0; ta_next(p, plan, &u, u0, u1, &s); ++n_seg) {
      const bool whole = s.n == s.nt;
      const size_t slot = ta_slot(s);
      const int N = (s.rows + 15) & ~15;
      // ---------------------------------------------------------- Q into its operand layout, and the rows' constants
      {
        constexpr int CH = D / 8, ROWS = TA_SOFT * 32 / CH;                // 16-byte pieces of a row; rows per pass
        const int c = threadIdx.x % CH, r_in = threadIdx.x / CH;
        const bool minus = p.scale < 0.f;                                 // the sign goes into q
        for (int r0 = 0; r0 < N; r0 += 2 * ROWS) {
          uint4 raw[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = r0 + i * ROWS + r_in;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (r < s.rows) {
              const int rk = s.rb * p.block + r, di = rk / p.group, hg = rk - di * p.group;
              raw[i] = *reinterpret_cast<const uint4*>(p.q + (size_t)(s.row0 + di) * p.ldq + (s.h * p.group + hg) * D + 8 * c);
              if (c == 0) {
                s_mask[r] = ta_mask(p, s.row0 + di, di, s.m);
                s_out[r] = whole ? (long long)(s.row0 + di) * p.ldo + (s.h * p.group + hg) * D : (long long)(slot * p.block + r) * D;
              }
            } else if (c == 0 && r < N) {
              s_mask[r] = 0;
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = r0 + i * ROWS + r_in;
            uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            float f = fabsf(p.scale) * 1.4426950408889634f;
            if constexpr (RAW16) {
#pragma unroll
              for (int y = 0; y < 4; ++y) w[y] ^= minus ? 0x80008000u : 0u;
            } else {
              float e[8], mx = 0.f;
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                e[2 * y] = __uint_as_float(w[y] << 16);
                e[2 * y + 1] = __uint_as_float(w[y] & 0xffff0000u);
                mx = fmaxf(mx, fmaxf(fabsf(e[2 * y]), fabsf(e[2 * y + 1])));
              }
#pragma unroll
              for (int off = CH / 2; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
              const int ex = scale_exponent(mx);
              const float up = minus ? -pow2_exact(ex) : pow2_exact(ex);
              f *= pow2_exact(-ex);
#pragma unroll
              for (int y = 0; y < 8; ++y) e[y] *= up;
#pragma unroll
              for (int y = 0; y < 4; ++y) w[y] = BITS == 4 ? ta_pack(e[y], e[y + 4], false) : ta_pack(e[2 * y], e[2 * y + 1], false);
            }
            if (r < N) {
              *reinterpret_cast<uint4*>(s_q + (c >> 3) * (NB * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
              if (c == 0) {
                float* fr = reinterpret_cast<float*>(&s_fr[r / 2]);
                fr[r & 1] = f;
                fr[2 + (r & 1)] = 0.f;
                s_unset[r] = true;
              }
            }
          }
        }
        fence_proxy_async_smem();
        if (threadIdx.x == 0) s_all_set = 0;
        named_bar_sync(3, TA_SOFT * 32);
        if (threadIdx.x == 0) mbar_arrive(&q_full);
      }
      bool ok = true;
      // ---------------------------------------------------------- tiles
      for (int j = (group ^ n0) & 1; j < s.n; j += 2) {
        const uint32_t n_tile = n0 + j, turn = n_tile >> 1;
        const uint32_t sbuf = tmem + TA_S + NB * (n_tile % Sh::SB) + lanes, pbuf = smem_u32(s_p) + group * Sh::P;
        const int t0 = (s.tile0 + j) * TA_TILE, back = t0 + t - s.len;   // the token's place among the drafts
        const bool masked = t0 + TA_TILE > s.len;
        ok = ta_wait(&s_full[n_tile % Sh::SB], (n_tile / Sh::SB) & 1, abort_v, ERR_TIMEOUT_FULL);
        if (ok && turn > 0) ok = ta_wait(&pv_done[group], (turn - 1) & 1, abort_v, ERR_TIMEOUT_FULL);   // P is free
        tc05_fence_after();
        // Does row r see this token?  Without branches, here and below: a branch per row would keep the rows' chains of
        // load, multiply-add, exponential and rounding from overlapping (47 cycles a row against 6).
        auto seen = [&](int r) -> bool { return (back < 0) | ((back < 64) & ((uint32_t)(s_mask[r] >> (back & 63)) & 1u)); };
        // the tile's weights into P; true if some visible score has outgrown its row's reference
        auto weigh_tile = [&](auto is_masked) -> bool {
          constexpr bool MASKED = decltype(is_masked)::value;
          float most = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < N; c += 32) {
            uint32_t v[32];
            tmem_ld32(sbuf + c, v);
            const uint32_t row = pbuf + (c >> 6) * (TA_TILE * 128) + t * 128;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              if (hf && c + 16 >= N) break;
              uint32_t w[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const int r = c + 16 * hf + 2 * x;
                const float4 fr = s_fr[r / 2];
                const float2 z = __ffma2_rn(make_float2(__uint_as_float(v[16 * hf + 2 * x]), __uint_as_float(v[16 * hf + 2 * x + 1])),
                                            make_float2(fr.x, fr.y), make_float2(fr.z, fr.w));
                float2 e = make_float2(ta_exp2(z.x), ta_exp2(z.y));
                if constexpr (MASKED) {
                  const bool s0 = seen(r), s1 = seen(r + 1);
                  most = ta_max3(most, s0 ? z.x : -INFINITY, s1 ? z.y : -INFINITY);
                  e.x = s0 ? e.x : 0.f;
                  e.y = s1 ? e.y : 0.f;
                } else {
                  most = ta_max3(most, z.x, z.y);
                }
                w[x] = ta_pack(e.x, e.y, RAW16);
              }
#pragma unroll
              for (int y = 0; y < 2; ++y)
                sts128(row + (((((c & 63) >> 3) + 2 * hf + y) ^ (t & 7)) << 4), w[4 * y], w[4 * y + 1], w[4 * y + 2], w[4 * y + 3]);
            }
          }
          return most > Sh::GROW;
        };
        auto weigh = [&]() -> bool { return masked ? weigh_tile(std::true_type{}) : weigh_tile(std::false_type{}); };
        // until every row has a reference, tiles go the long way
        const int version = s_version;
        const bool known = s_all_set;
        bool grown = false;
        if (ok && known) grown = weigh();
        if (ok && n_tile > 0) ok = ta_wait(&checked[group ^ 1], ((n_tile - 1) >> 1) & 1, abort_v, ERR_TIMEOUT_FULL);
        const bool all_known = s_all_set;
        if (ok && all_known && (!known || version != s_version)) grown = weigh();
        fence_proxy_async_smem();
        tc05_fence_before();
        if (lane == 0) s_failed[warp] = !ok;
        if (ta_any<128>(bar, grown || !ok || !all_known)) {
          if (s_failed[4 * group] || s_failed[4 * group + 1] || s_failed[4 * group + 2] || s_failed[4 * group + 3]) {
            ok = false;                                 // all four warps leave together
            break;
          }
          // O and L are to be rescaled: the product of the tile before has to be over (the one before that is)
          if (j > 0) ok = ta_wait(&pv_done[group ^ 1], ((n_tile - 1) >> 1) & 1, abort_v, ERR_TIMEOUT_FULL);
          tc05_fence_after();
          // ------------------------------------------------------ new references
          auto maxima = [&](auto is_masked) {
#pragma unroll 1
            for (int c = 0; c < N; c += 16) {
              float v[16];
              tmem_ld16(sbuf + c, v);
              int mine = 0;
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                float z = v[x] * reinterpret_cast<const float*>(&s_fr[(c + x) / 2])[x & 1];
                if constexpr (decltype(is_masked)::value) z = seen(c + x) ? z : -INFINITY;
                const int top = __reduce_max_sync(0xffffffffu, ta_key(z));
                mine = lane == x ? top : mine;
              }
              if (lane < 16) s_key[gw][c + lane] = mine;
            }
          };
          if (masked) maxima(std::true_type{}); else maxima(std::false_type{});
          named_bar_sync(bar, 128);
          bool late = false;
          if (t < N) {
            const float top = ta_unkey(max(max(s_key[0][t], s_key[1][t]), max(s_key[2][t], s_key[3][t])));
            float* nref = &reinterpret_cast<float*>(&s_fr[t / 2])[2 + (t & 1)];
            float fix = 1.f;
            if (s_unset[t]) {                           // no weight so far: O and L are zero (or NaN, which stays)
              s_unset[t] = !(top > -INFINITY);          // nothing visible yet (or a NaN, which needs no reference)
              if (!s_unset[t]) *nref = Sh::BIAS - top;
            } else if (top + *nref > Sh::GROW) {
              const float now = Sh::BIAS - top;
              fix = ta_exp2(now - *nref);
              *nref = now;
            }
            s_fix[t] = fix;
            late = s_unset[t] && t < s.rows;
          }
          late = ta_any<128>(bar, late);
          if (t == 0) {
            s_all_set = !late;
            ++s_version;
          }
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < 2 * N; c += 16) {       // O, then L
              const int r = c < N ? c : c - N;
              const uint32_t at = tmem + lanes + (c < N ? TA_O : TA_L) + r;
              float o[16];
              tmem_ld16(at, o);
              uint32_t x[16];
#pragma unroll
              for (int y = 0; y < 16; ++y) x[y] = __float_as_uint(o[y] * s_fix[r + y]);
              tmem_st16(at, x);
            }
            tmem_st_wait();
          }
          weigh();
          fence_proxy_async_smem();
          tc05_fence_before();
          if (lane == 0) s_failed[warp] = !ok;
          if (ta_any<128>(bar, !ok)) {
            ok = false;
            break;
          }
        }
        if (t == 0) {
          mbar_arrive(&p_full[group]);
          mbar_arrive(&s_free[n_tile % Sh::SB]);
          mbar_arrive(&checked[group]);
        }
      }
      n0 += s.n;
      // ---------------------------------------------------------- the end of the run: lane = element, column = row
      if (ok) ok = ta_wait(&run_done, n_seg & 1, abort_v, ERR_TIMEOUT_FULL);
      if (ta_any<256>(3, !ok)) break;                   // both groups go on together or not at all
      tc05_fence_after();
      // codes of 4 bits stand at another position inside each 8 elements
      const int d = BITS == 4 ? (t & ~7) + ((t & 7) >> 1) + 4 * (t & 1) : t;
      auto finish = [&](auto is_whole) {
#pragma unroll 1
        for (int c = 16 * group; c < N; c += 32) {
          float o[16], l[16];
          tmem_ld16(tmem + lanes + TA_O + c, o);
          tmem_ld16(tmem + lanes + TA_L + c, l);
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const bool there = c + x < s.rows;
            if constexpr (decltype(is_whole)::value) {
              const float val = l[x] == 0.f ? 0.f : __fdividef(o[x], l[x]);   // a row that saw nothing is zero
              if (there) p.out[s_out[c + x] + d] = __float2bfloat16_rn(val);
            } else {
              if (there) p.partial[s_out[c + x] + d] = o[x];
            }
          }
          if constexpr (!decltype(is_whole)::value) {
            float mine = 0.f;                           // every lane has every row's weight: lane x keeps row x's
#pragma unroll
            for (int x = 0; x < 16; ++x) mine = lane == x ? l[x] : mine;
            if (t < 16 && c + t < s.rows) {
              // the reference that the sums stand at (a row without weight has none)
              p.stats[2 * slot * p.block + c + t] =
                  mine == 0.f ? -INFINITY : -reinterpret_cast<const float*>(&s_fr[(c + t) / 2])[2 + (t & 1)];
              p.stats[(2 * slot + 1) * p.block + c + t] = mine;
            }
          }
        }
      };
      if (t < D) {
        if (whole) finish(std::true_type{}); else finish(std::false_type{});
      }
      if (s_bad[n_seg % TA_FLAGS]) {
        // V held infinities or NaN in drafted tokens, which were left out of the products: the rows that see one get it here
        named_bar_sync(3, TA_SOFT * 32);                // the values to add to are written
#pragma unroll 1
        for (int r = group; t < D && r < s.rows; r += 2) {
          float extra = 0.f;
#pragma unroll 1
          for (int i = 0; i < s.m; ++i) {
            const int pos = s.len + i;
            if (!(s_mask[r] >> i & 1) || pos < s.tile0 * TA_TILE || pos >= (s.tile0 + s.n) * TA_TILE) continue;
            const int page = p.table[(size_t)s.b * p.table_pages + (pos >> p.c.page_shift)];
            if ((unsigned)page >= (unsigned)p.c.n_pages) continue;
            const float v = ta_cache_value<BITS>(p.c.p.v, p.c.p.vs, p.c.p.vb,
                                                 kv_token(p.c, page, s.h, pos & ((1 << p.c.page_shift) - 1)), D, t);
            if (!isfinite(v)) extra += v;
          }
          if (extra == 0.f) continue;
          if (whole) p.out[s_out[r] + t] = __float2bfloat16_rn(__bfloat162float(p.out[s_out[r] + t]) + extra);
          else p.partial[s_out[r] + t] += extra;
        }
      }
      tc05_fence_before();
      named_bar_sync(3, TA_SOFT * 32);                  // the rows' constants and O are free for the next run
      tc05_fence_after();
      if (threadIdx.x == 0) s_bad[n_seg % TA_FLAGS] = 0;
    }
  }
  tc05_fence_before();
  __syncthreads();
  if (warp == Sh::MMA) {
    tc05_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int BITS, int NB>
static cudaError_t launch_rows(const TreeAttnParams& p, cudaStream_t s) {
  using Sh = TaShape<D, BITS, NB>;
  const cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<D, BITS, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(p.grid), dim3(Sh::THREADS), Sh::SMEM, s, attr);
  return cudaLaunchKernelEx(&cfg, tree_attn_kernel<D, BITS, NB>, p);
}
template <int D, int BITS>
static cudaError_t launch_bits(const TreeAttnParams& p, cudaStream_t s) {
  return p.block == 64 ? launch_rows<D, BITS, 64>(p, s) : launch_rows<D, BITS, 128>(p, s);
}

cudaError_t launch_tree_attn(const TreeAttnParams& p, cudaStream_t s) {
  if (p.c.dim == 128)
    return p.c.bits == 16 ? launch_bits<128, 16>(p, s) : (p.c.bits == 8 ? launch_bits<128, 8>(p, s) : launch_bits<128, 4>(p, s));
  return p.c.bits == 16 ? launch_bits<64, 16>(p, s) : (p.c.bits == 8 ? launch_bits<64, 8>(p, s) : launch_bits<64, 4>(p, s));
}

}  // namespace sv
