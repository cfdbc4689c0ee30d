// RMS norm of each query and key head with the position rotation in the same
// pass (mlx-dspark wiki page, "Architecture": the step between the q | k | v
// projection and the cache; the pages give no layer internals).
//
//   x <- x / sqrt(mean(x^2) + eps) * w,   (x_i, x_j) <- (x_i cos a - x_j sin a, x_j cos a + x_i sin a)
//
// Bound by memory for prompts and by launch latency for a drafted block: each
// q and k element is read once and written once.  A lane owns 8 adjacent
// elements of a head (one 16-byte access each way), a head is D / 8 adjacent
// lanes of a warp (rounded up to a power of two), the mean is a shuffle tree,
// and the rotation's partner chunk - rotary_dim / 2 elements away - comes from
// another lane by shuffle, so a head's values never leave registers.
//
// A warp is on its own: it takes some heads of one row, makes the row's sines and
// cosines while its first loads are in flight (each lane a few frequencies, handed
// over through the warp's piece of shared memory) and holds those of its chunk in
// registers over all its heads.  No barrier joins warps.  Measured: 4093 rows of 56 heads of 128, 64 of them rotated in adjacent
// pairs, 23.5 us (5.0 TB/s of the 6.8 that a copy reaches; 77 us with a CTA a row and fp64 angles); 40 heads rotated in halves of all
// 128 elements 22.0 us (3.8 TB/s: cosines, sines, weights and 40 values do not fit 64 registers, 120 bytes a thread are spilled); 8 rows
// of 40 heads 2.1 us.
//
// Angles.  position * inv_freq reaches 1e6 radians, where one fp32 ulp is 0.06
// rad, and fp64 is slow here.  In units of 2^-64 turns the product is one of integers,
// and whole turns fall off at the top: 64 bits of inv_freq / 2 pi times the position,
// mod 2^64, off by at most |position| * 2^-63 turns for any frequency.  Its upper 32 bits, as a float
// (2^-26 turns), go to sincospif.
#include "sv_kv.cuh"

namespace sv {

struct RopeParams {
  const __nv_bfloat16* in[2];   // q, k
  __nv_bfloat16* out[2];
  const __nv_bfloat16* w[2];
  int ld_in[2], ld_out[2], heads[2];
  int dim, half, lanes;         // half = rotary_dim / 2; lanes per head
  int rows, split, batches[2];  // warps of a row; batches of AHEAD passes of 32 / lanes heads
  float eps, mean;              // mean = 1 / dim
  const int32_t* positions;
  const float* inv_freq;
};

constexpr int ROPE_WARPS = 4;
constexpr int ROPE_CTAS = 8;   // per SM: 64 registers a thread
constexpr int ROPE_MAX_HALF = 128;
constexpr int ROPE_AHEAD = 4;  // chunks a lane has in flight
constexpr int ROPE_FILL = 32;  // warps per SM that a call asks for

// Pairs that rotate together.
enum RopePairs { ROPE_NONE, ROPE_HALVES, ROPE_ADJACENT };

__device__ __forceinline__ uint4 load_chunk(const __nv_bfloat16* p, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
  uint4 r;
  r.x = u[0] | ((uint32_t)u[1] << 16);
  r.y = u[2] | ((uint32_t)u[3] << 16);
  r.z = u[4] | ((uint32_t)u[5] << 16);
  r.w = u[6] | ((uint32_t)u[7] << 16);
  return r;
}

// 2^96 / 2 pi: the turns in a radian, its first 64 bits and the next 32.
constexpr unsigned long long RADIAN_HIGH = 2935890503282001226ull, RADIAN_LOW = 2131351028ull;

// (cos, sin) of position * f.  f = m * 2^(e - 23) with a 24-bit m; from 2^24 on (and for
// infinity and NaN) no phase is left in it and the result is NaN.
__device__ __forceinline__ float2 rope_turn(int position, float f) {
  const uint32_t u = __float_as_uint(f);
  const int e = (int)((u >> 23) & 255) - 127, shift = 23 - e;
  const uint64_t m = (u & 0x7fffff) | (e > -127 ? 0x800000u : 0u);
  const uint64_t main = m * RADIAN_HIGH, lo = main + (m * RADIAN_LOW >> 32), hi = __umul64hi(m, RADIAN_HIGH) + (lo < main);
  uint64_t c = 0;               // the product hi:lo in units of 2^(e - 87) turns, shifted right to 2^-64 (by 0 to 150)
  if (shift <= 0) c = lo;
  else if (shift < 64) c = (lo >> shift) | (hi << (64 - shift));
  else if (shift < 128) c = hi >> (shift - 64);
  const uint64_t turns = (u >> 31 ? 0 - c : c) * (uint64_t)(int64_t)position;
  float sn, cs;
  sincospif((float)(int32_t)(turns >> 32) * (shift < 0 ? __int_as_float(0x7fffffff) : 4.656612873077393e-10f), &sn, &cs);
  return make_float2(cs, sn);
}

// Batches are q's, then k's: none has heads of both, so one weight and one pair of pointers serve a batch.
template <int PAIRS, bool NORM, bool VEC, int AHEAD>
__global__ void __launch_bounds__(32 * ROPE_WARPS, ROPE_CTAS) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(16) float s_cos[ROPE_WARPS][ROPE_MAX_HALF], s_sin[ROPE_WARPS][ROPE_MAX_HALF];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int task = blockIdx.x * ROPE_WARPS + warp;
  const int row = (int)((uint32_t)task / (uint32_t)p.split), part = task - row * p.split;
  if (row >= p.rows) return;    // whole warps: what follows is warp-wide
  const int L = p.lanes, j = lane & (L - 1), per = 32 / L;  // j: chunk of the head
  const int batches = p.batches[0] + p.batches[1];
  const int first = (int)((uint32_t)(part * batches) / (uint32_t)p.split);
  const int end = (int)((uint32_t)((part + 1) * batches) / (uint32_t)p.split);
  const bool in_head = j * 8 < p.dim;
  const int hc = p.half / 8;
  const bool low = j < hc, turned = j * 8 < 2 * p.half;
  float c[8], s[8];             // of this lane's chunk; adjacent pairs use 4
  float w[8];
  for (int batch = first; batch < end; ++batch) {
    const int t = batch >= p.batches[0], heads = p.heads[t];
    const int h0 = (batch - (t ? p.batches[0] : 0)) * AHEAD * per + lane / L;
    const __nv_bfloat16* src = p.in[t] + (size_t)row * p.ld_in[t] + h0 * p.dim + j * 8;
    __nv_bfloat16* dst = p.out[t] + (size_t)row * p.ld_out[t] + h0 * p.dim + j * 8;
    const int hop = per * p.dim;
    uint4 raw[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      raw[i] = make_uint4(0, 0, 0, 0);
      if (in_head && h0 + i * per < heads) raw[i] = load_chunk(src + i * hop, VEC);
    }
    if (NORM && (batch == first || batch == p.batches[0])) {
      uint4 w4 = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);  // ones
      if (p.w[t] && in_head) w4 = load_chunk(p.w[t] + j * 8, VEC);
      const uint32_t u[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = __uint_as_float(e & 1 ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
    }
    if (PAIRS != ROPE_NONE && batch == first) {
      const int position = p.positions[row];
      for (int f = lane; f < p.half; f += 64) {  // two at a time: their latencies overlap
        const int g = f + 32 < p.half ? f + 32 : f;
        const float ff = p.inv_freq[f], fg = p.inv_freq[g];
        const float2 cf = rope_turn(position, ff), cg = rope_turn(position, fg);
        s_cos[warp][f] = cf.x;
        s_sin[warp][f] = cf.y;
        s_cos[warp][g] = cg.x;
        s_sin[warp][g] = cg.y;
      }
      __syncwarp();
      // adjacent: chunk j holds pairs 4j..; halves: chunk j of either half the frequencies 8j..
      const int f0 = !turned ? 0 : (PAIRS == ROPE_ADJACENT ? 4 * j : 8 * (low ? j : j - hc));
      const float sign = PAIRS == ROPE_HALVES && low ? -1.f : 1.f;
#pragma unroll
      for (int e = 0; e < (PAIRS == ROPE_ADJACENT ? 4 : 8); e += 4) {
        const float4 a = *reinterpret_cast<const float4*>(&s_cos[warp][f0 + e]);
        const float4 b = *reinterpret_cast<const float4*>(&s_sin[warp][f0 + e]);
        c[e] = a.x, c[e + 1] = a.y, c[e + 2] = a.z, c[e + 3] = a.w;
        s[e] = sign * b.x, s[e + 1] = sign * b.y, s[e + 2] = sign * b.z, s[e + 3] = sign * b.w;
      }
    }
    float x[AHEAD][8], ss[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      ss[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[i][e] = __uint_as_float(e & 1 ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
        if (NORM) ss[i] = fmaf(x[i][e], x[i][e], ss[i]);
      }
    }
    if (NORM) {
      for (int off = L / 2; off; off >>= 1) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], off);
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const float r = rsqrtf(fmaf(ss[i], p.mean, p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * r * w[e];
      }
    }
    if (PAIRS == ROPE_ADJACENT) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = x[i][2 * e], b = x[i][2 * e + 1];
          x[i][2 * e] = turned ? a * c[e] - b * s[e] : a;
          x[i][2 * e + 1] = turned ? b * c[e] + a * s[e] : b;
        }
      }
    }
    if (PAIRS == ROPE_HALVES) {
      const int from = (lane & ~(L - 1)) + (low ? j + hc : (turned ? j - hc : j));
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xffffffffu, x[i][e], from);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = turned ? x[i][e] * c[e] + o[e] * s[e] : x[i][e];
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (in_head && h0 + i * per < heads) {
        if (VEC) {
          uint4 o4;
          __nv_bfloat162* o2 = reinterpret_cast<__nv_bfloat162*>(&o4);
#pragma unroll
          for (int e = 0; e < 4; ++e) o2[e] = __floats2bfloat162_rn(x[i][2 * e], x[i][2 * e + 1]);
          *reinterpret_cast<uint4*>(dst + i * hop) = o4;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[i * hop + e] = __float2bfloat16_rn(x[i][e]);
        }
      }
    }
  }
}

}  // namespace sv

using namespace sv;

extern "C" int sv_qk_norm_rope(const uint16_t* q, int ldq, const uint16_t* k, int ldk, int rows, int n_q_heads,
                               int n_kv_heads, int head_dim, int norm, const uint16_t* q_weight,
                               const uint16_t* k_weight, float eps, const int32_t* positions, const float* inv_freq,
                               int rotary_dim, int interleaved, uint16_t* q_out, int ldqo, uint16_t* k_out, int ldko,
                               void* stream) {
  if (rows < 0 || rows > (1 << 20)) return fail(SV_EINVAL, "rows must be in [0, 2^20] (got %d)", rows);
  if (n_q_heads < 1 || n_q_heads > 4096 || n_kv_heads < 0 || n_kv_heads > 4096)
    return fail(SV_EINVAL, "head counts out of range (got %d, %d)", n_q_heads, n_kv_heads);
  if (head_dim < 8 || head_dim > 256 || head_dim % 8)
    return fail(SV_EUNSUPPORTED, "head_dim must be a multiple of 8 up to 256 (got %d)", head_dim);
  if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16)
    return fail(SV_EUNSUPPORTED, "rotary_dim must be a multiple of 16 up to head_dim (got %d)", rotary_dim);
  if (!q || !q_out || (n_kv_heads && (!k || !k_out))) return fail(SV_EINVAL, "q, k and their outputs must be non-null");
  if (rotary_dim && (!positions || !inv_freq)) return fail(SV_EINVAL, "a rotation needs positions and inv_freq");
  const long long qw = (long long)n_q_heads * head_dim, kw = (long long)n_kv_heads * head_dim;
  if (ldq < qw || ldqo < qw || (n_kv_heads && (ldk < kw || ldko < kw)))
    return fail(SV_EINVAL, "strides must be >= heads * head_dim");
  if ((q == q_out && ldq != ldqo) || (n_kv_heads && k == k_out && ldk != ldko))
    return fail(SV_EINVAL, "an in-place call needs equal strides");
  if (norm && !(eps >= 0.f)) return fail(SV_EINVAL, "eps must be >= 0");
  if (!aligned(q, 2) || !aligned(q_out, 2) || !aligned(k, 2) || !aligned(k_out, 2) || !aligned(positions, 4) ||
      !aligned(inv_freq, 4) || !aligned(q_weight, 2) || !aligned(k_weight, 2))
    return fail(SV_EINVAL, "a pointer is not aligned to its element");
  if (!rows) return SV_OK;
  RopeParams p = {};
  const uint16_t* in[2] = {q, k};
  uint16_t* out[2] = {q_out, k_out};
  const uint16_t* w[2] = {q_weight, k_weight};
  const int li[2] = {ldq, ldk}, lo[2] = {ldqo, ldko}, hs[2] = {n_q_heads, n_kv_heads};
  bool vec = true;              // 16-byte accesses allowed
  for (int t = 0; t < 2; ++t) {
    p.in[t] = reinterpret_cast<const __nv_bfloat16*>(in[t]);
    p.out[t] = reinterpret_cast<__nv_bfloat16*>(out[t]);
    p.w[t] = reinterpret_cast<const __nv_bfloat16*>(w[t]);
    p.ld_in[t] = li[t];
    p.ld_out[t] = lo[t];
    p.heads[t] = hs[t];
    if (hs[t])
      vec = vec && aligned(in[t], 16) && aligned(out[t], 16) && (!w[t] || aligned(w[t], 16)) && li[t] % 8 == 0 && lo[t] % 8 == 0;
  }
  p.dim = head_dim;
  p.half = rotary_dim / 2;
  p.lanes = 1;
  while (p.lanes * 8 < head_dim) p.lanes *= 2;
  p.eps = eps;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.rows = rows;
  p.mean = 1.f / (float)head_dim;
  const int sms = device_sm_count();
  if (sms <= 0) return fail(SV_ECUDA, "no CUDA device");
  // Few rows: one pass per warp, for parallelism.  Many: ROPE_AHEAD of them at once, for bytes in flight.
  const int per = 32 / p.lanes, passes[2] = {(n_q_heads + per - 1) / per, (n_kv_heads + per - 1) / per};
  const bool many = vec && passes[0] >= ROPE_AHEAD && (long long)rows * (passes[0] + passes[1]) >= ROPE_FILL * ROPE_AHEAD * sms;
  const int ahead = many ? ROPE_AHEAD : 1;
  for (int t = 0; t < 2; ++t) p.batches[t] = (passes[t] + ahead - 1) / ahead;
  // Warps of a row: as many as give each SM ROPE_FILL of them, at most one a batch.
  p.split = (ROPE_FILL * sms + rows - 1) / rows;
  if (p.split > p.batches[0] + p.batches[1]) p.split = p.batches[0] + p.batches[1];
  const long long tasks = (long long)rows * p.split;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)((tasks + ROPE_WARPS - 1) / ROPE_WARPS)), dim3(32 * ROPE_WARPS), 0,
                                      static_cast<cudaStream_t>(stream), attr);
  using Kernel = void (*)(RopeParams);
#define SV_ROPE(PAIRS, NORM) \
  {rope_kernel<PAIRS, NORM, false, 1>, rope_kernel<PAIRS, NORM, true, 1>, rope_kernel<PAIRS, NORM, true, ROPE_AHEAD>}
  static constexpr Kernel kernels[3][2][3] = {{SV_ROPE(ROPE_NONE, false), SV_ROPE(ROPE_NONE, true)},
                                              {SV_ROPE(ROPE_HALVES, false), SV_ROPE(ROPE_HALVES, true)},
                                              {SV_ROPE(ROPE_ADJACENT, false), SV_ROPE(ROPE_ADJACENT, true)}};
#undef SV_ROPE
  const int pairs = !rotary_dim ? ROPE_NONE : (interleaved ? ROPE_ADJACENT : ROPE_HALVES);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernels[pairs][norm != 0][many ? 2 : vec], p);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "norm and rotation launch");
}
