// Building blocks of the attention kernels on the 5th-generation tensor cores: a ring of operand tiles, waits of whole warps, and the
// warps that turn codes into fp16 operands.
#pragma once

#include "sv_tc05.cuh"
#include "tree_attn.cuh"

namespace sv {

constexpr int TA_TILE = 128;                       // tokens per tile
constexpr int TA_TEAM = 4;                         // warps of a transforming team

// One operand tile of codes as the transforming warps need it: where each 16 tokens' codes, scales and biases are (past the
// end, the cache's first tokens stand in: nothing comes of them), and what is odd about it.
struct TaPiece {
  const uint8_t* codes[TA_TILE / 16];
  const __half* scales[TA_TILE / 16];
  const __half* biases[TA_TILE / 16];
  int valid;                    // tokens of the tile before the end of the sequence; 0: the work has ended
  int drafted;                  // first drafted token of the tile (TA_TILE and more: none)
  int is_v;
  int flag;                     // the segment's flag in s_bad
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

// Codes that one CTA alone reads are not kept in L2; those of a prefix are read by others too.
template <bool ONCE>
__device__ __forceinline__ uint4 ta_load_codes(const uint4* p) { return ONCE ? __ldcs(p) : __ldcg(p); }

// Codes -> fp16 operands, by warp `tw` of transforming team `team`, until a piece without tokens.  DRAFTS: tiles may hold drafted tokens.
template <int D, int BITS, int TEAMS, int OPS, bool DRAFTS>
__device__ __forceinline__ void ta_transform(uint8_t* ops, uint64_t* op_full, uint64_t* op_empty, TaPiece* pieces, uint64_t* piece_full,
                                             uint64_t* piece_empty, int* s_bad, volatile int* abort_v, int team, int tw, int lane) {
  // A team takes every TEAMS-th operand tile, a warp 32 of its tokens.  Codes come from global memory in 16-byte
  // loads, LPT neighbouring lanes per token; the registers of a step are loaded for the team's next tile as soon
  // as they are used, so the loads of a whole tile are always on their way.
  constexpr int ROWB = D * BITS / 8, LPT = ROWB / 16, TPS = 32 / LPT, PERT = 128 / BITS;  // codes per 16 bytes
  constexpr int NCH = PERT / 8, G = D / GROUP;      // 16-byte operand chunks a lane makes per step; groups per token
  // The lane's 16 bytes of a token, and its token of a step: where 8 neighbouring lanes would meet the same banks with their
  // operand chunks - the two 64-element halves of a token lie 16 KB apart - they take each other's tokens.
  const int part = lane & (LPT - 1);
  const int sub = LPT == 8 ? lane / LPT ^ part >> 2 : (NCH == 4 && LPT == 4 ? lane / LPT ^ (part >> 1) << 1 : lane / LPT);
  const int grp = part * PERT / GROUP, c0 = (part * PERT / 8) & 7;
  const uint32_t pick = G == 2 && grp ? 0x3232 : 0x1010;
  // Where this lane's chunks go in its first row; the rows of later steps differ in the swizzle by one bit at most.
  uint32_t to[NCH];
#pragma unroll
  for (int y = 0; y < NCH; ++y)
    to[y] = (part * PERT / 64) * (TA_TILE * 128) + (32 * tw + sub) * 128 + (((c0 + y) ^ (sub & 7)) << 4);
  const int t = 32 * tw + lane;                       // this lane's token of a tile
  TaRing<OPS> ring;
  TaRing<TA_PIECES> ahead, here;
  ring.next(team);
  ahead.next(team);
  here.next(team);
  uint4 raw[LPT];
  uint32_t sc = 0, bi = 0;                          // scales and biases of this lane's token (two groups, or one)
  const uint8_t* at[2] = {};                        // the warp's two 16-token halves
  const int lane_at = sub * ROWB + part * 16;
  bool live = true;
  // the next tile's addresses, scales and biases
  auto locate = [&]() -> bool {
    if (!ta_wait(&piece_full[ahead.slot], ahead.phase, abort_v, ERR_TIMEOUT_FULL)) return false;
    const TaPiece& x = pieces[ahead.slot];
    live = x.valid > 0;
    if (live) {
      at[0] = x.codes[2 * tw] + lane_at;
      at[1] = x.codes[2 * tw + 1] + lane_at;
      const __half *ps = x.scales[2 * tw + lane / 16] + (lane & 15) * G, *pb = x.biases[2 * tw + lane / 16] + (lane & 15) * G;
      if constexpr (G == 2) {
        sc = *reinterpret_cast<const uint32_t*>(ps);
        bi = *reinterpret_cast<const uint32_t*>(pb);
      } else {
        sc = *reinterpret_cast<const unsigned short*>(ps);
        bi = *reinterpret_cast<const unsigned short*>(pb);
      }
    }
    ahead.next(TEAMS);
    return true;
  };
  auto fetch = [&] {
#pragma unroll
    for (int i = 0; i < LPT; ++i) raw[i] = ta_load_codes<DRAFTS>(reinterpret_cast<const uint4*>(at[i * TPS / 16] + (i * TPS % 16) * ROWB));
  };
#pragma unroll
  for (int i = 0; i < LPT; ++i) raw[i] = make_uint4(0, 0, 0, 0);
  bool ok = locate();
  if (ok && live) fetch();
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
      if (DRAFTS && odd) s_bad[x.flag] = 1;
    }
    uint32_t even[NCH], odd[NCH];                   // in the rows of even steps, and of odd ones
#pragma unroll
    for (int y = 0; y < NCH; ++y) {
      even[y] = to[y] + ring.slot * (TA_TILE * D * 2);
      odd[y] = even[y] ^ ((TPS & 7) << 4);
    }
#pragma unroll
    for (int i = 0; i < LPT; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      const uint32_t s1 = __shfl_sync(0xffffffffu, sv, i * TPS + sub), b1 = __shfl_sync(0xffffffffu, bv, i * TPS + sub);
      const uint32_t sp = __byte_perm(s1, 0, pick), bp = __byte_perm(b1, 0, pick);
      const __half2 s2 = *reinterpret_cast<const __half2*>(&sp), b2 = *reinterpret_cast<const __half2*>(&bp);
      uint32_t o[64 / BITS];
#pragma unroll
      for (int y = 0; y < 4; ++y) ta_dequant<BITS>(w[y], s2, b2, o + y * (16 / BITS));
#pragma unroll
      for (int y = 0; y < NCH; ++y)
        *reinterpret_cast<uint4*>(ops + (i & 1 ? odd[y] : even[y]) + i * TPS * 128) = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
    }
    fence_proxy_async_smem();  // the tensor cores read these writes through the async proxy
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&op_full[ring.slot]);
      mbar_arrive(&piece_empty[here.slot]);
    }
    ring.next(TEAMS);
    here.next(TEAMS);
    ok = locate();
    if (!ok) break;
    if (live) fetch();
  }
}

}  // namespace sv
