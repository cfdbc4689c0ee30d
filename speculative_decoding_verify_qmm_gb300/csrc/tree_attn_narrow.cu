// Tree attention of few rows (drafted rows x query heads per key head), with warp-level matrix instructions.
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - max)
//
// Bound by instructions over codes in blocks of 16 rows (some 470 a warp for 16 tokens, half of them codes to fp16; issue in 63 % of
// cycles), by latency in blocks of 32 (two warps to a scheduler, issue in 34 %) and for short contexts: a cached byte meets 16 to 64 multiply-adds, far below what warp-level MMA
// gives.  A warp owns every W-th step of 16 tokens of the CTA's run, with its own ring of cp.async stages in shared memory, its
// own running maximum, weight and sums in registers, and no barrier of the CTA until the run ends, where the warps' sums are
// joined in warp order.
//
// Over codes the sums' registers decide.  One row tile of 16: two warps are a team, each makes the weights of its own 16 tokens,
// hands them to the other through shared memory, and sums half of the head over the tokens of both: 16 warps of 128 registers,
// four to a scheduler.  Two row tiles: 8 warps, and a warp takes two steps at once where it can, so that two chains overlap.
// (Teams for two row tiles spill: 207 us against 193; 16 warps without teams join in two rounds: 11.6 us for one row against 10.1.)
//
// Measured (32 query and 8 key heads of 128): one row over 2048 tokens, 8-bit, 9.5 us; 8 rows over 16384 tokens, 8-bit, 23.2 us
// (1.5 TB/s); 48 requests of 1 to 5 rows, up to 12007 tokens, 4-bit, 158 us (2.6 TB/s of the 6.8 that a copy reaches).
//
// Codes become MMA operands in registers, without a second trip through shared memory.  S = Q K^T: the contraction may run
// over a head's elements in any order, so the lane that holds column q of a token's k-slices takes whole 16-byte pieces of
// its codes and Q is laid out to match.  O += P V: P's accumulator layout is the A operand's; V's pairs (two tokens, one
// element) come from byte shuffles of the two tokens' words, and the output's columns are numbered so that a lane owns a
// contiguous piece of a V row.  fp16 s * c + b with the exact code (half an fp16 step); Q enters as fp16 scaled by a power of
// two per row; 16-bit caches go through bf16 MMA as they are.
//
// MT row tiles of 16 per warp.
#include <type_traits>

#include "tree_attn.cuh"

namespace sv {

constexpr int TN_STEP = 16;  // tokens per warp step

template <int D, int BITS, int MT>
struct TnShape {
  static constexpr int TEAM = BITS != 16 && MT == 1 ? 2 : 1;                    // warps that share their tokens' weights
  static constexpr int PAIR = BITS != 16 && MT == 2 ? 2 : 1;                    // steps that a warp takes at once, if it can
  static constexpr int W = 8 * TEAM;                                            // warps
  static constexpr int THREADS = 32 * W, BLOCK = 16 * MT;
  static constexpr int ROWB = D * BITS / 8, G = D / GROUP;
  static constexpr int SIDE = BITS == 16 ? 0 : TN_STEP * G * 2;                 // one array of scales or biases
  static constexpr int STAGE = 2 * TN_STEP * ROWB + 4 * SIDE;
  static constexpr int QBYTES = MT * (D / 16) * 512;
  static constexpr int WEIGHTS = TEAM == 2 ? W * MT * 512 : 0;                   // handed over within a team
  static constexpr int LD = D == 128 ? 144 : 72;                                // floats per row of a joined tile (conflict-free)
  static constexpr int TILE = 16 * LD * 4, JOIN = 8 * MT * TILE;
  static constexpr int BUDGET = 218 * 1024 - QBYTES - WEIGHTS;
  static constexpr int FIT = BUDGET / (W * STAGE);
  static constexpr int NST = FIT > 8 ? 8 : FIT;
  static constexpr int RING = W * NST * STAGE;
  static constexpr int SMEM = QBYTES + WEIGHTS + (RING > JOIN ? RING : JOIN);             // the join's tiles lie in the drained ring
  static_assert(NST >= 2 * PAIR && MT <= W, "stages, and a warp for each row tile of Q");
  // as in the kernel for many rows: the largest weight's exponent when the reference is set, and what it may grow to
  static constexpr float BIAS = BITS == 16 ? -30.f : 5.f, GROW = BITS == 16 ? -15.f : 15.f;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool BF16>
__device__ __forceinline__ void tn_mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// (biased - OFFSET) * s + b, with fp16 OFFSET
template <int OFFSET = 0x6400>  // 1024
__device__ __forceinline__ uint32_t tn_fma(uint32_t biased, uint32_t s2, uint32_t b2) {
  const __half2 offset = __half2half2(__ushort_as_half((unsigned short)OFFSET));
  const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&s2), __hsub2(*reinterpret_cast<const __half2*>(&biased), offset),
                            *reinterpret_cast<const __half2*>(&b2));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// The 4-bit codes at bit AT of both halves of c: in the low bits of 1024, or 4 bits higher in those of 64, they are added to it.
template <int AT>
__device__ __forceinline__ uint32_t tn_code4(uint32_t c, uint32_t s2, uint32_t b2) {
  return AT == 0 ? tn_fma<0x6400>((c & 0x000f000fu) | 0x64006400u, s2, b2) : tn_fma<0x5400>((c & 0x00f000f0u) | 0x54005400u, s2, b2);
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], int at, const uint8_t* p) {
  if constexpr (N >= 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[at] = v.x; w[at + 1] = v.y; w[at + 2] = v.z; w[at + 3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
__device__ __forceinline__ uint32_t lds32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint32_t lds16(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }

// Which of the lane's elements are the four of k-slice kk: (b0 low, b0 high, b1 low, b1 high).
template <int BITS>
__device__ __forceinline__ int tn_k_pick(int kk, int i) {
  if (BITS != 4) return 4 * kk + i;
  return 8 * (kk / 2) + 2 * (kk & 1) + (i >> 1) + 4 * (i & 1);
}
// Element of output column `col` of n-tile nt: a lane's share of a V row (of a team's warp: of half a row) is contiguous.
template <int D, int BITS, int TEAM>
__device__ __forceinline__ int tn_v_elem(int half, int nt, int col) {
  if (D == 128 && BITS == 16) return (nt >> 3) * 64 + 8 * col + (nt & 7);
  return TEAM == 1 ? (D / 8) * col + nt : half * (D / 2) + (D / 16) * col + nt;
}

// Of the two warps of a team: a barrier, and whether a lane of either says so.
__device__ __forceinline__ void team_sync(int team) { asm volatile("bar.sync %0, 64;" ::"r"(team + 1) : "memory"); }
__device__ __forceinline__ bool team_any(int team, bool mine) {
  int any;
  asm volatile(
      "{\n .reg .pred a, b;\n setp.ne.s32 a, %1, 0;\n bar.red.or.pred b, %2, 64, a;\n selp.s32 %0, 1, 0, b;\n}"
      : "=r"(any)
      : "r"((int)mine), "r"(team + 1)
      : "memory");
  return any != 0;
}

template <int D, int BITS, int MT>
__global__ void __launch_bounds__(TnShape<D, BITS, MT>::THREADS, 1) tree_attn_narrow_kernel(const __grid_constant__ TreeAttnParams p) {
  using Sh = TnShape<D, BITS, MT>;
  constexpr bool RAW16 = BITS == 16;
  constexpr int ROWB = Sh::ROWB, CPR = ROWB / 16, G = Sh::G, NST = Sh::NST, KK = D / 16, NTW = D / 8 / Sh::TEAM;
  constexpr int KW = D * BITS / 128;                         // 32-bit words of a lane's share of a K row
  constexpr int VB = NTW * BITS / 8, VW = (VB + 3) / 4;      // bytes and words of its share of a V row, or of the warp's half of it
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ TaPlan plan;
  __shared__ float s_f[Sh::BLOCK], s_max[Sh::W][16 * MT], s_sum[Sh::W][16 * MT], s_top[Sh::W][16 * MT];
  __shared__ long long s_out[Sh::BLOCK];                   // where each row of the block is written (elements)
  __shared__ uint64_t s_mask[Sh::BLOCK];
  __shared__ int s_odd;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int team = warp / Sh::TEAM, half = Sh::TEAM == 2 ? warp & 1 : 0;   // half of the head's elements in O
  uint4* const qf = reinterpret_cast<uint4*>(smem);         // [MT][KK][32]
  uint4* const weights = reinterpret_cast<uint4*>(smem + Sh::QBYTES);   // [W][MT][32]
  uint8_t* const ring = smem + Sh::QBYTES + Sh::WEIGHTS + warp * NST * Sh::STAGE;
  const uint32_t ring_a = smem_u32(ring);
  float* const tiles = reinterpret_cast<float*>(smem + Sh::QBYTES + Sh::WEIGHTS);

  const TaShare share = ta_begin(p, &plan);
  const long long u0 = share.u0, u1 = share.u1;
  const int pm = (1 << p.c.page_shift) - 1;

  TaSeg s = share.s;
  long long u = share.u;
  for (bool more = share.more; more; more = ta_next(p, plan, &u, u0, u1, &s)) {
    // ------------------------------------------------------------ the ring
    const int mts = s.rows > 16 ? MT : 1;                                   // row tiles with rows
    const int first = s.tile0 << (TA_UNIT_SHIFT - 4), all = (s.total + TN_STEP - 1) / TN_STEP;   // in steps
    const int run = all - first < s.n << (TA_UNIT_SHIFT - 4) ? all - first : s.n << (TA_UNIT_SHIFT - 4);
    const int own = run > warp ? (run - warp + Sh::W - 1) / Sh::W : 0;      // this warp's
    const int lead = Sh::TEAM == 2 ? warp & ~1 : warp;                      // its team's: the last may be the lead's alone
    const int steps = run > lead ? (run - lead + Sh::W - 1) / Sh::W : 0;
    int pages = 0;                                                          // lane i: the page of step (base + i)
    auto load_pages = [&](int base) {
      const int k = base + lane;
      pages = 0;
      if (k < own) {
        const int t = (first + warp + k * Sh::W) * TN_STEP;
        pages = p.table[(size_t)s.b * p.table_pages + (t >> p.c.page_shift)];
      }
    };
    load_pages(0);
    auto issue = [&](int k) {
      if (k < own) {
        if (k && !(k & 31)) load_pages(k);
        int page = __shfl_sync(0xffffffffu, pages, k & 31);
        if ((unsigned)page >= (unsigned)p.c.n_pages) {
          raise_error(ERR_BAD_INPUT);
          page = 0;                                                          // stay inside the arrays: the result is undefined
        }
        const int t = (first + warp + k * Sh::W) * TN_STEP;
        const size_t tok = kv_token(p.c, page, s.h, t & pm);
        const uint32_t st = ring_a + (k % NST) * Sh::STAGE;
        const uint8_t *ks = p.c.p.k + tok * ROWB, *vs = p.c.p.v + tok * ROWB;
#pragma unroll
        for (int i = 0; i < CPR / 2; ++i) {
          // chunk c of token r; the place of a chunk in its row keeps the lanes that read together on different banks
          const int id = i * 32 + lane, r = id / CPR, c = id % CPR;
          const int fk = CPR >= 8 ? (r & 1) << 2 : 0;
          const int fv = CPR >= 8 ? ((r >> 1) & 3) << 1 : (CPR == 4 ? (r >> 1) & 3 : 0);
          cp_async16(st + r * ROWB + ((c ^ fk) << 4), ks + id * 16);
          cp_async16(st + TN_STEP * ROWB + r * ROWB + ((c ^ fv) << 4), vs + id * 16);
        }
        if constexpr (!RAW16) {
          constexpr int SC = Sh::SIDE / 16;                                  // chunks of one array
          if (lane < 4 * SC) {
            const int a = lane / SC, c = lane % SC;
            const __half* src = (a == 0 ? p.c.p.ks : (a == 1 ? p.c.p.kb : (a == 2 ? p.c.p.vs : p.c.p.vb))) + tok * G;
            cp_async16(st + 2 * TN_STEP * ROWB + lane * 16, reinterpret_cast<const uint8_t*>(src) + c * 16);
          }
        }
      }
      cp_async_commit();
    };
    // ------------------------------------------------------------ Q, as A operands
    if (threadIdx.x == 0) s_odd = 0;
    const bool minus = p.scale < 0.f;                                       // the sign goes into q
    const int t = warp;                                                     // a warp a row tile
    const bool has_q = t < MT;
    // this lane's share of two rows: the elements that its share of a K row meets
    constexpr int PE = D * BITS >= 512 ? 128 / BITS : D / 4, NP = D / 4 / PE;
    uint4 raw[2][D / 32];
    bool real[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = 16 * t + 8 * i + g;
      real[i] = has_q && k < s.rows;
      const int r = s.rb * p.block + k, di = real[i] ? ta_by_group(p, r) : 0, hg = real[i] ? r - di * p.group : 0;
      const __nv_bfloat16* src = p.q + (size_t)(s.row0 + di) * p.ldq + (s.h * p.group + hg) * D;
#pragma unroll
      for (int c = 0; c < NP; ++c)
#pragma unroll
        for (int y = 0; y < PE / 8; ++y)
          raw[i][c * (PE / 8) + y] = real[i] ? *reinterpret_cast<const uint4*>(src + (4 * c + q) * PE + 8 * y) : make_uint4(0, 0, 0, 0);
    }
    uint64_t mask = 0;                                 // of row 16 t + 8 q + g, kept by the lanes with q < 2
    if (has_q && q < 2 && 16 * t + 8 * q + g < s.rows) {
      const int di = ta_by_group(p, s.rb * p.block + 16 * t + 8 * q + g);
      mask = ta_mask(p, s.row0 + di, di, s.m);
    }
    // (asked for before the ring's copies, which would hold these loads up)
    // The warps that convert Q fill their rings afterwards, but for two stages: the others' copies keep the memory busy.
#pragma unroll 1
    for (int turn = 0, next = 0; turn < 2; ++turn) {
#pragma unroll 1
      for (; next < (turn || !has_q || NST < 4 ? NST - 1 : 2); ++next) issue(next);
      if (turn == 0) {
        if (has_q) {
          float up[2] = {minus ? -1.f : 1.f, minus ? -1.f : 1.f};
          float f[2];
          f[0] = f[1] = ta_score_factor(p.scale, 0);
          auto elem = [&](int i, int e) -> float {           // the e-th of the share
            const uint4 v = raw[i][e / 8];
            const uint32_t w = (e / 2) % 4 == 0 ? v.x : ((e / 2) % 4 == 1 ? v.y : ((e / 2) % 4 == 2 ? v.z : v.w));
            return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
          };
          if constexpr (!RAW16) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float mx = 0.f;
#pragma unroll
              for (int e = 0; e < D / 4; ++e) mx = fmaxf(mx, fabsf(elem(i, e)));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
              const int ex = ta_query_exponent(mx);
              up[i] *= pow2_exact(ex);
              f[i] = ta_score_factor(p.scale, ex);
            }
          }
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) {
            float x[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[i][e] = elem(i, tn_k_pick<BITS>(kk, e)) * up[i];
            qf[(t * KK + kk) * 32 + lane] = make_uint4(ta_pack(x[0][0], x[0][1], RAW16), ta_pack(x[1][0], x[1][1], RAW16),
                                                       ta_pack(x[0][2], x[0][3], RAW16), ta_pack(x[1][2], x[1][3], RAW16));
          }
          if (q < 2) {
            const int k = 16 * t + 8 * q + g, r = s.rb * p.block + k, di = ta_by_group(p, r);
            s_f[k] = q ? f[1] : f[0];
            s_mask[k] = mask;
            s_out[k] = s.n == s.nt ? (long long)(s.row0 + di) * p.ldo + (s.h * p.group + r - di * p.group) * D
                                   : (long long)(ta_slot(s) * p.block + k) * D;
          }
        }
        __syncthreads();
      }
    }
    // ------------------------------------------------------------ this warp's rows
    float o[MT][NTW][4], f[MT][2], nref[MT][2], lim[MT][2], sum[MT][2];   // nref: minus the reference, lim: how far a score may outgrow it
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int n = 0; n < NTW; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][n][e] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = 16 * m + 8 * i + g;
        f[m][i] = s_f[k];
        nref[m][i] = 0.f;
        lim[m][i] = -INFINITY;                           // no reference yet
        sum[m][i] = 0.f;
      }
    }
    const uint4* const qw = qf + lane;
    // Steps k .. k + NS - 1, the first from token t0 on; of each warp of a team.  Whether they are masked and how many row tiles they
    // have are fixed at compile time: branches inside would keep the independent chains of conversions and products from
    // overlapping.
    auto step = [&](int k, int t0, auto is_masked, auto row_tiles, auto at_once) {
      constexpr bool masked = decltype(is_masked)::value;
      constexpr int MS = decltype(row_tiles)::value, NS = decltype(at_once)::value;
      static_assert(NS == 1 || (!masked && Sh::TEAM == 1), "masks and teams: one step at a time");
      const uint8_t* st[NS];
#pragma unroll
      for (int x = 0; x < NS; ++x) st[x] = ring + ((k + x) % NST) * Sh::STAGE;
      // ------------------------------------------------------------ S = Q K^T
      float sc[NS][MS][2][4];
#pragma unroll
      for (int x = 0; x < NS; ++x)
#pragma unroll
        for (int m = 0; m < MS; ++m)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[x][m][n][e] = 0.f;
      {
        uint32_t w[NS][2][KW], s2[NS][2][2], b2[NS][2][2];                   // [token half][group of the piece]
#pragma unroll
        for (int x = 0; x < NS; ++x)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int r = 8 * n + g;
            const uint8_t* row = st[x] + r * ROWB;
            if constexpr (KW >= 4) {
#pragma unroll
              for (int c = 0; c < KW / 4; ++c) lds_words(w[x][n], 4 * c, row + (((4 * c + q) ^ (CPR >= 8 ? (r & 1) << 2 : 0)) << 4));
            } else {
              lds_words(w[x][n], 0, row + q * 8);
            }
            if constexpr (!RAW16) {
              const uint8_t* side = st[x] + 2 * TN_STEP * ROWB + r * (2 * G);
              if constexpr (G == 2) {
                const uint32_t a = lds32(side), b = lds32(side + Sh::SIDE);
                if constexpr (KW == 8) {                                       // piece 0 is group 0, piece 1 group 1
                  s2[x][n][0] = __byte_perm(a, 0, 0x1010); s2[x][n][1] = __byte_perm(a, 0, 0x3232);
                  b2[x][n][0] = __byte_perm(b, 0, 0x1010); b2[x][n][1] = __byte_perm(b, 0, 0x3232);
                } else {                                                       // one piece: group q / 2
                  s2[x][n][0] = s2[x][n][1] = __byte_perm(a, 0, q & 2 ? 0x3232 : 0x1010);
                  b2[x][n][0] = b2[x][n][1] = __byte_perm(b, 0, q & 2 ? 0x3232 : 0x1010);
                }
              } else {
                s2[x][n][0] = s2[x][n][1] = __byte_perm(lds16(side), 0, 0x1010);
                b2[x][n][0] = b2[x][n][1] = __byte_perm(lds16(side + Sh::SIDE), 0, 0x1010);
              }
            }
          }
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          uint4 a[MS];
#pragma unroll
          for (int m = 0; m < MS; ++m) a[m] = qw[(m * KK + kk) * 32];
#pragma unroll
          for (int x = 0; x < NS; ++x)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              uint32_t b0, b1;
              if constexpr (RAW16) {
                b0 = w[x][n][2 * kk];
                b1 = w[x][n][2 * kk + 1];
              } else {
                const int gp = KW == 8 ? kk / 4 : 0;
                if constexpr (BITS == 8) {
                  b0 = tn_fma(__byte_perm(w[x][n][kk], 0x64646464u, 0x4140), s2[x][n][gp], b2[x][n][gp]);
                  b1 = tn_fma(__byte_perm(w[x][n][kk], 0x64646464u, 0x4342), s2[x][n][gp], b2[x][n][gp]);
                } else {
                  const uint32_t c = w[x][n][kk / 2] >> (8 * (kk & 1));
                  b0 = tn_code4<0>(c, s2[x][n][gp], b2[x][n][gp]);
                  b1 = tn_code4<4>(c, s2[x][n][gp], b2[x][n][gp]);
                }
              }
#pragma unroll
              for (int m = 0; m < MS; ++m) tn_mma<RAW16>(sc[x][m][n], a[m], b0, b1);
            }
        }
      }
      // ------------------------------------------------------------ weights
      uint32_t see[MS][2];                                                   // visible tokens of the step, per row half
      float top[MS][2];
      bool grown = false;
      auto shown = [&](int m, int n, int e) { return see[m][e >> 1] >> (8 * n + 2 * q + (e & 1)) & 1; };
#pragma unroll
      for (int m = 0; m < MS; ++m) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (masked) {
            const int d = t0 - s.len;                                        // drafted index of the step's first token
            const uint64_t bits = s_mask[16 * m + 8 * i + g];
            see[m][i] = d <= -32 ? 0xffffu : (d < 0 ? ((1u << -d) - 1) | (uint32_t)(bits << -d) : (d < 64 ? (uint32_t)(bits >> d) : 0u));
          }
          top[m][i] = -INFINITY;
        }
#pragma unroll
        for (int x = 0; x < NS; ++x)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) top[m][e >> 1] = fmaxf(top[m][e >> 1], !masked || shown(m, n, e) ? sc[x][m][n][e] : -INFINITY);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[m][i] = top[m][i] == -INFINITY ? top[m][i] : top[m][i] * f[m][i];
          grown |= top[m][i] + nref[m][i] > lim[m][i];                       // (nothing visible: never)
        }
      }
      if (Sh::TEAM == 2 ? team_any(team, grown) : __any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int m = 0; m < MS; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            top[m][i] = fmaxf(top[m][i], __shfl_xor_sync(0xffffffffu, top[m][i], 1));
            top[m][i] = fmaxf(top[m][i], __shfl_xor_sync(0xffffffffu, top[m][i], 2));
            if (Sh::TEAM == 2 && q == 0) s_top[warp][16 * m + 8 * i + g] = top[m][i];
          }
        if (Sh::TEAM == 2) team_sync(team);
#pragma unroll
        for (int m = 0; m < MS; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (Sh::TEAM == 2) top[m][i] = fmaxf(top[m][i], s_top[warp ^ 1][16 * m + 8 * i + g]);
            const bool move = top[m][i] + nref[m][i] > lim[m][i];            // alike in the row's lanes
            const float now = move ? Sh::BIAS - top[m][i] : nref[m][i];
            const float fix = lim[m][i] == -INFINITY ? 1.f : ta_exp2(now - nref[m][i]);   // no weight so far: nothing to rescale
            lim[m][i] = move ? Sh::GROW : lim[m][i];
            nref[m][i] = now;
            sum[m][i] *= fix;
#pragma unroll
            for (int n = 0; n < NTW; ++n) {
              o[m][n][2 * i] *= fix;
              o[m][n][2 * i + 1] *= fix;
            }
          }
      }
      if (Sh::TEAM == 2) issue(k + NST - 1);                                 // its stage: both warps are done with the step before
      uint4 pa[NS * Sh::TEAM][MS];
#pragma unroll
      for (int x = 0; x < NS; ++x)
#pragma unroll
        for (int m = 0; m < MS; ++m) {
          float w[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = e >> 1;
              const float y = ta_exp2(fmaf(sc[x][m][n][e], f[m][i], nref[m][i]));
              w[n][e] = !masked || shown(m, n, e) ? y : 0.f;
              sum[m][i] += w[n][e];
            }
          pa[x][m] = make_uint4(ta_pack(w[0][0], w[0][1], RAW16), ta_pack(w[0][2], w[0][3], RAW16), ta_pack(w[1][0], w[1][1], RAW16),
                                ta_pack(w[1][2], w[1][3], RAW16));
        }
      if constexpr (Sh::TEAM == 2) {
#pragma unroll
        for (int m = 0; m < MS; ++m) weights[(warp * MT + m) * 32 + lane] = pa[0][m];
        team_sync(team);
#pragma unroll
        for (int m = 0; m < MS; ++m) pa[1][m] = weights[((warp ^ 1) * MT + m) * 32 + lane];
      }
      // ------------------------------------------------------------ O += P V
#pragma unroll
      for (int x = 0; x < NS * Sh::TEAM; ++x) {                              // of a team: this warp's tokens, then the other's
        const int hop = warp & 1 ? -1 : 1;
        const uint8_t* const sv = Sh::TEAM == 2 ? st[0] + x * hop * NST * Sh::STAGE : st[x % NS];
        const int tx = t0 + x * (Sh::TEAM == 2 ? hop : Sh::W) * TN_STEP;
        uint32_t w[4][VW], s2[2], b2[2];                                     // tokens 2q, 2q + 1, 2q + 8, 2q + 9
        const int valid = s.total - tx, drafted = s.len - tx;
        bool odd = false;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int r = 2 * q + (z & 1) + 8 * (z >> 1);
          const uint8_t* row = sv + TN_STEP * ROWB + r * ROWB;
          const int fv = CPR >= 8 ? ((r >> 1) & 3) << 1 : (CPR == 4 ? (r >> 1) & 3 : 0);
          if constexpr (VB >= 16) {
#pragma unroll
            for (int c = 0; c < VB / 16; ++c) lds_words(w[z], 4 * c, row + (((8 * c + g) ^ fv) << 4));
          } else {
            const int at = (half * 8 + g) * VB;                              // bytes before the lane's share
            const uint8_t* from = row + (((at >> 4) ^ fv) << 4) + (at & 15);
            if constexpr (VB == 2) w[z][0] = lds16(from);
            else lds_words(w[z], 0, from);
          }
          if constexpr (RAW16 && masked) {
            // Rows past the end are zeroed (their weight is 0, and 0 * NaN would not be); so are a drafted row's
            // infinities and NaN, which only rows that see it may get (added in when the run is written).
#pragma unroll
            for (int y = 0; y < VW; ++y) {
              if (r >= valid) {
                w[z][y] = 0;
              } else if (r >= drafted) {
                if ((w[z][y] & 0x7f80u) == 0x7f80u) { w[z][y] &= 0xffff0000u; odd = true; }
                if ((w[z][y] & 0x7f800000u) == 0x7f800000u) { w[z][y] &= 0x0000ffffu; odd = true; }
              }
            }
          }
        }
        if constexpr (!RAW16) {
          const uint8_t* side = sv + 2 * TN_STEP * ROWB + 2 * Sh::SIDE + (G == 2 ? (Sh::TEAM == 2 ? half : g >> 2) * 2 : 0);
#pragma unroll
          for (int y = 0; y < 2; ++y) {                                      // token pairs
            uint32_t a[2], b[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int r = 2 * q + z + 8 * y;
              a[z] = lds16(side + r * (2 * G));
              b[z] = lds16(side + r * (2 * G) + Sh::SIDE);
              if constexpr (masked) {                                        // as above, a group at a time
                const bool wild = ta_half_bad(a[z]) | ta_half_bad(b[z]), off = (r >= valid) | ((r >= drafted) & wild);
                odd |= off & (r < valid);
                a[z] = off ? 0 : a[z];
                b[z] = off ? 0 : b[z];
              }
            }
            s2[y] = a[0] | a[1] << 16;
            b2[y] = b[0] | b[1] << 16;
          }
        }
        if constexpr (masked) {
          if (odd) s_odd = 1;
        }
#pragma unroll
        for (int n = 0; n < NTW; ++n) {
          uint32_t b[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t *A = w[2 * y], *B = w[2 * y + 1];
            if constexpr (RAW16) {
              b[y] = __byte_perm(A[n / 2], B[n / 2], n & 1 ? 0x7632 : 0x5410);
            } else if constexpr (BITS == 8) {
              const uint32_t c = __byte_perm(A[n / 4], B[n / 4], n & 2 ? 0x7362 : 0x5140);
              b[y] = tn_fma(__byte_perm(c, 0x64646464u, n & 1 ? 0x4342 : 0x4140), s2[y], b2[y]);
            } else {
              const uint32_t c = __byte_perm(A[n / 8], B[n / 8], n & 4 ? 0x7632 : 0x5410) >> (8 * (n >> 1 & 1));
              b[y] = n & 1 ? tn_code4<4>(c, s2[y], b2[y]) : tn_code4<0>(c, s2[y], b2[y]);
            }
          }
#pragma unroll
          for (int m = 0; m < MS; ++m) tn_mma<RAW16>(o[m][n], pa[x][m], b[0], b[1]);
        }
      }
    };
    const int plain = s.len >> 4;                                            // steps before this see committed tokens only
    for (int k = 0; k < steps;) {
      using One = std::integral_constant<int, 1>;
      using All = std::integral_constant<int, MT>;
      const int at = first + warp + k * Sh::W, t0 = at * TN_STEP;
      const bool two = Sh::PAIR == 2 && k + 1 < steps && at + Sh::W < plain;
      if (two) cp_async_wait<NST - Sh::PAIR - 1>();
      else cp_async_wait<NST - 2>();
      __syncwarp();                                                          // every lane's copies of the stages have landed
      if (two) {
        if constexpr (Sh::PAIR == 2) {
          using Two = std::integral_constant<int, 2>;
          if (mts == 1) step(k, t0, std::false_type{}, One{}, Two{});
          else step(k, t0, std::false_type{}, All{}, Two{});
        }
      } else if (Sh::PAIR == 2 || (Sh::TEAM == 2 ? at | 1 : at) >= plain) {  // (beside pairs, a lone step is not worth its own code)
        if (mts == 1) step(k, t0, std::true_type{}, One{}, One{});
        else step(k, t0, std::true_type{}, All{}, One{});
      } else {
        if (mts == 1) step(k, t0, std::false_type{}, One{}, One{});
        else step(k, t0, std::false_type{}, All{}, One{});
      }
      if (Sh::TEAM == 1) {
        __syncwarp();                                                        // the stages may be overwritten
        issue(k + NST - 1);
        if (two) issue(k + NST);
      }
      k += two ? 2 : 1;
    }
    // ------------------------------------------------------------ the warps' sums meet
    cp_async_wait<0>();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = sum[m][i];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (q == 0) {
          s_max[warp][16 * m + 8 * i + g] = lim[m][i] == -INFINITY ? -INFINITY : -nref[m][i];
          s_sum[warp][16 * m + 8 * i + g] = x;
        }
      }
    __syncthreads();
    const bool whole = s.n == s.nt, odd = s_odd != 0;
    const size_t slot = ta_slot(s);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = 16 * m + 8 * i + g;
        float most = -INFINITY, weight = 0.f;            // over the warps, each of the row's lanes a quarter of them
#pragma unroll
        for (int x = 0; x < Sh::W; x += 4) most = fmaxf(most, s_max[x + q][k]);
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const float base = most == -INFINITY ? 0.f : most;
#pragma unroll
        for (int x = 0; x < Sh::W; x += 4) weight += s_sum[x + q][k] * ta_exp2(s_max[x + q][k] - base);
        weight += __shfl_xor_sync(0xffffffffu, weight, 1);
        weight += __shfl_xor_sync(0xffffffffu, weight, 2);
        const float own = ta_exp2(s_max[warp][k] - base), factor = whole ? (weight == 0.f ? 0.f : own / weight) : own;
#pragma unroll
        for (int n = 0; n < NTW; ++n) {
          o[m][n][2 * i] *= factor;
          o[m][n][2 * i + 1] *= factor;
        }
        if (!whole && warp == 0 && q == 0 && k < s.rows) {
          p.stats[(2 * slot) * p.block + k] = most;
          p.stats[(2 * slot + 1) * p.block + k] = weight;
        }
      }
    constexpr int LD = Sh::LD;
    // a lane's sums of one row tile, in element order
    auto put = [&](int m, float* tile) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int n = 0; n < NTW; n += 4) {
            const int d = tn_v_elem<D, BITS, Sh::TEAM>(half, n, 2 * q + e);
            float4* at = reinterpret_cast<float4*>(tile + (8 * i + g) * LD + d + (d >> 5) * 4);
            const int c = 2 * i + e;
            *at = make_float4(o[m][n][c], o[m][n + 1][c], o[m][n + 2][c], o[m][n + 3][c]);
          }
    };
#pragma unroll
    for (int m = 0; m < MT; ++m) put(m, tiles + (8 * m + team) * (Sh::TILE / 4));
    __syncthreads();
    {
      constexpr int QUADS = D / 4;
      for (int idx = threadIdx.x; idx < 16 * MT * QUADS; idx += Sh::THREADS) {
        const int k = idx / QUADS, d0 = 4 * (idx % QUADS);
        if (k >= s.rows) continue;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const float4 t = *reinterpret_cast<const float4*>(tiles + (8 * (k / 16) + y) * (Sh::TILE / 4) + (k % 16) * LD + d0 + (d0 >> 5) * 4);
          a.x += t.x; a.y += t.y; a.z += t.z; a.w += t.w;
        }
        if (odd) {
          // V held infinities or NaN in drafted tokens, which were left out of the products: the rows that see one get it
          const int r = s.rb * p.block + k, di = ta_by_group(p, r);
          const uint64_t see = ta_mask(p, s.row0 + di, di, s.m);
          float* e = reinterpret_cast<float*>(&a);
#pragma unroll 1
          for (int i = 0; i < 4 * s.m; ++i) {
            const int pos = s.len + i / 4;
            if (!(see >> (i / 4) & 1) || pos < s.tile0 << TA_UNIT_SHIFT || pos >= (s.tile0 + s.n) << TA_UNIT_SHIFT) continue;
            const int page = p.table[(size_t)s.b * p.table_pages + (pos >> p.c.page_shift)];
            if ((unsigned)page >= (unsigned)p.c.n_pages) continue;
            const float v = ta_cache_value<BITS>(p.c.p.v, p.c.p.vs, p.c.p.vb, kv_token(p.c, page, s.h, pos & pm), D, d0 + i % 4);
            if (!isfinite(v)) e[i % 4] += v;
          }
        }
        if (whole) {
          __nv_bfloat162 o2[2] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w)};
          *reinterpret_cast<uint2*>(p.out + s_out[k] + d0) = *reinterpret_cast<uint2*>(o2);
        } else {
          *reinterpret_cast<float4*>(p.partial + s_out[k] + d0) = a;
        }
      }
      __syncthreads();
    }
  }
}

template <int D, int BITS, int MT>
static cudaError_t launch_narrow(const TreeAttnParams& p, cudaStream_t s) {
  using Sh = TnShape<D, BITS, MT>;
  const cudaError_t e =
      cudaFuncSetAttribute(tree_attn_narrow_kernel<D, BITS, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(p.grid), dim3(Sh::THREADS), Sh::SMEM, s, attr);
  return cudaLaunchKernelEx(&cfg, tree_attn_narrow_kernel<D, BITS, MT>, p);
}
template <int D, int BITS>
static cudaError_t launch_narrow_rows(const TreeAttnParams& p, cudaStream_t s) {
  return p.block == 16 ? launch_narrow<D, BITS, 1>(p, s) : launch_narrow<D, BITS, 2>(p, s);
}

cudaError_t launch_tree_attn_narrow(const TreeAttnParams& p, cudaStream_t s) {
  if (p.c.dim == 128)
    return p.c.bits == 16 ? launch_narrow_rows<128, 16>(p, s)
                          : (p.c.bits == 8 ? launch_narrow_rows<128, 8>(p, s) : launch_narrow_rows<128, 4>(p, s));
  return p.c.bits == 16 ? launch_narrow_rows<64, 16>(p, s)
                        : (p.c.bits == 8 ? launch_narrow_rows<64, 8>(p, s) : launch_narrow_rows<64, 4>(p, s));
}

}  // namespace sv
