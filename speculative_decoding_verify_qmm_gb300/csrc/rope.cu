// RMS norm of each query and key head with the position rotation in the same
// pass (mlx-dspark wiki page, "Architecture": the step between the q | k | v
// projection and the cache; the pages give no layer internals).
//
//   x <- x / sqrt(mean(x^2) + eps) * w,   (x_i, x_j) <- (x_i cos a - x_j sin a, x_j cos a + x_i sin a)
//
// Bound by memory for prompts and by launch latency for a drafted block: each
// q and k element is read once and written once.  A thread owns 8 adjacent
// elements of a head (one 16-byte access each way), a head is D / 8 adjacent
// lanes of a warp (rounded up to a power of two), the mean is a shuffle tree,
// and the rotation's partner chunk - rotary_dim / 2 elements away - comes from
// another lane by shuffle, so a head's values never leave registers.  The
// sines and cosines of a row are made once per CTA, in shared memory, while the
// first loads are in flight.
//
// Angles: position * inv_freq reaches 1e6 radians, where one fp32 ulp is 0.06
// rad.  It is formed in fp64 in units of turns, its whole turns are dropped, and
// the rest (at most half a turn, error 2^-25 turns) goes to sincospif.
#include "sv_kv.cuh"

namespace sv {

struct RopeParams {
  const __nv_bfloat16* in[2];   // q, k
  __nv_bfloat16* out[2];
  const __nv_bfloat16* w[2];
  int ld_in[2], ld_out[2], heads[2];
  bool vec_in[2], vec_out[2];   // 16-byte accesses allowed
  int dim, half, lanes;         // half = rotary_dim / 2; lanes per head
  bool norm, interleaved;
  float eps;
  const int32_t* positions;
  const float* inv_freq;
};

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_AHEAD = 4;  // chunks a thread loads before it computes

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

__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 s_cs[128];
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, tid = threadIdx.x;
  const int L = p.lanes, j = tid & (L - 1);              // chunk of the head
  const int per = ROPE_THREADS / L, slots = per * gridDim.y;
  const int total = p.heads[0] + p.heads[1];
  const bool live = j * 8 < p.dim;
  // every thread of the CTA makes the same number of passes (the shuffles are warp-wide)
  for (int base = blockIdx.y * per; base < total; base += slots * ROPE_AHEAD) {
    uint4 raw[ROPE_AHEAD];
#pragma unroll
    for (int i = 0; i < ROPE_AHEAD; ++i) {
      const int h = base + i * slots + tid / L;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (live && h < total) {
        const int t = h >= p.heads[0], hh = t ? h - p.heads[0] : h;
        raw[i] = load_chunk(p.in[t] + (size_t)row * p.ld_in[t] + hh * p.dim + j * 8, p.vec_in[t]);
      }
    }
    if (base == blockIdx.y * per) {
      for (int f = tid; f < p.half; f += ROPE_THREADS) {
        const double turns = (double)p.positions[row] * (double)p.inv_freq[f] * 0.15915494309189533577;
        float sn, cs;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
        s_cs[f] = make_float2(cs, sn);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < ROPE_AHEAD; ++i) {
      if (base + i * slots >= total) break;              // uniform over the CTA
      const int h = base + i * slots + tid / L;
      const int t = h >= p.heads[0], hh = t ? h - p.heads[0] : h;
      float x[8];
      const __nv_bfloat162* r2 = reinterpret_cast<const __nv_bfloat162*>(&raw[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __bfloat1622float2(r2[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
      if (p.norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
        for (int off = L / 2; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float r = rsqrtf(ss / (float)p.dim + p.eps);
        const __nv_bfloat16* w = p.w[t];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= r;
          if (w && live) x[e] *= __bfloat162float(w[j * 8 + e]);
        }
      }
      if (p.half) {
        if (p.interleaved) {
          if (j * 8 < 2 * p.half) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 cs = s_cs[4 * j + e];
              const float a = x[2 * e], b = x[2 * e + 1];
              x[2 * e] = a * cs.x - b * cs.y;
              x[2 * e + 1] = b * cs.x + a * cs.y;
            }
          }
        } else {
          const int hc = p.half / 8;                     // chunks of half the rotated part
          const bool low = j < hc, turned = j < 2 * hc;
          const int from = (tid & 31 & ~(L - 1)) + (low ? j + hc : (turned ? j - hc : j));
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xffffffffu, x[e], from);
          if (turned) {
            const int f0 = 8 * (low ? j : j - hc);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 cs = s_cs[f0 + e];
              x[e] = low ? x[e] * cs.x - o[e] * cs.y : x[e] * cs.x + o[e] * cs.y;
            }
          }
        }
      }
      if (live && h < total) {
        __nv_bfloat16* dst = p.out[t] + (size_t)row * p.ld_out[t] + hh * p.dim + j * 8;
        if (p.vec_out[t]) {
          uint4 o4;
          __nv_bfloat162* o2 = reinterpret_cast<__nv_bfloat162*>(&o4);
#pragma unroll
          for (int e = 0; e < 4; ++e) o2[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
          *reinterpret_cast<uint4*>(dst) = o4;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = __float2bfloat16_rn(x[e]);
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
  for (int t = 0; t < 2; ++t) {
    p.in[t] = reinterpret_cast<const __nv_bfloat16*>(in[t]);
    p.out[t] = reinterpret_cast<__nv_bfloat16*>(out[t]);
    p.w[t] = reinterpret_cast<const __nv_bfloat16*>(w[t]);
    p.ld_in[t] = li[t];
    p.ld_out[t] = lo[t];
    p.heads[t] = hs[t];
    p.vec_in[t] = aligned(in[t], 16) && li[t] % 8 == 0;
    p.vec_out[t] = aligned(out[t], 16) && lo[t] % 8 == 0;
  }
  p.dim = head_dim;
  p.half = rotary_dim / 2;
  p.lanes = 1;
  while (p.lanes * 8 < head_dim) p.lanes *= 2;
  p.norm = norm != 0;
  p.interleaved = interleaved != 0;
  p.eps = eps;
  p.positions = positions;
  p.inv_freq = inv_freq;
  // Few rows: one pass of heads per CTA, for parallelism.  Many: one CTA a row, so
  // that a row's sines and cosines (fp64, slow here) are made once.
  const int per = ROPE_THREADS / p.lanes, passes = (n_q_heads + n_kv_heads + per - 1) / per;
  const int sms = device_sm_count();
  if (sms <= 0) return fail(SV_ECUDA, "no CUDA device");
  const int split = rows >= 2 * sms ? 1 : passes;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3(rows, split), dim3(ROPE_THREADS), 0, static_cast<cudaStream_t>(stream), attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_kernel, p);
  return e == cudaSuccess ? SV_OK : cuda_fail(e, "norm and rotation launch");
}
