// Shared by the kernel of tree attention and the join: their parameters, how the work is dealt, and how a finished run of an item is
// written.
//
// Every (request, key head, block of rows) is an item of ceil(tokens / 128) units.  A unit's cost depends on the rows, and
// beginning an item costs a CTA as much as some units (its rows to load, the pipeline to fill, the sums to write); the items,
// in order, are dealt to the CTAs in equal contiguous shares of that cost.  Ragged lengths balance, and one long sequence
// fills the GPU.  A CTA that has an item whole writes the output; parts of an item leave fp32 sums (with their maximum and
// weight) in the workspace, and a second kernel joins them in CTA order.  Each CTA has at most two such parts: of the item
// that its share begins in, and of the one that it ends in.
#pragma once

#include "sv_kv.cuh"

namespace sv {

constexpr int TA_UNIT_SHIFT = 7;                   // log2 of the tokens dealt at once: a tile of the kernel

struct TreeAttnParams {
  CUtensorMap tk, tv;        // 16-bit caches: [pages * heads][page][dim], boxes of 64 x min(page, 128)
  KvCache c;
  RowMap map;
  const int32_t *kv_len, *table;
  int table_pages;
  const __nv_bfloat16* q; int ldq;
  int group;                 // query heads per key head
  uint32_t per_group;        // 2^20 / group, rounded up
  float scale;
  const uint64_t* mask;
  __nv_bfloat16* out; int ldo;
  float* partial;            // [2 * grid][block][dim] sums of the CTAs' unfinished items
  float* stats;              // [2 * grid][2][block]: their maximum (as an exponent of 2) and weight
  int grid;
  int block;                 // rows (drafted row x query head of the group) per item
  int cost[2];               // of a unit with up to 16 rows, and with more
  int begin_cost;            // of beginning an item
};

// What every CTA derives from the lengths: prefix sums of units.
struct TaPlan {
  long long pre[MAX_BATCH + 1];   // cost of the requests before b
  int items[MAX_BATCH + 1];       // their items (its first entry is not used)
  int len[MAX_BATCH];             // committed tokens, brought into the table's range
  int begin;                      // p.begin_cost, or nothing where the shares are too small to hold a second beginning
};

__host__ __device__ __forceinline__ int ta_blocks(int rows, int block) { return (rows + block - 1) / block; }

__device__ __forceinline__ int ta_cost(const TreeAttnParams& p, int m) { return p.cost[m * p.group > 16]; }

// By one warp; `real` false: with lengths of zero, which reads nothing.
__device__ __forceinline__ void ta_plan(const TreeAttnParams& p, TaPlan* plan, bool real, bool report) {
  const int lane = threadIdx.x & 31;
  const RowMap& map = p.map;
  const long long cap = (long long)p.table_pages << p.c.page_shift;   // at least every request's rows (checked by the host)
  long long run = 0;             // of the units' cost
  int items = 0;
  for (int b0 = 0; b0 < map.B; b0 += 32) {
    const int b = b0 + lane;
    long long inc = 0;
    int n = 0;
    if (b < map.B) {
      const int m = map.offs[b + 1] - map.offs[b];
      long long len = real ? p.kv_len[b] : 0;
      if (m && (len < 0 || len + m > cap)) {
        if (report) raise_error(ERR_BAD_INPUT);
        len = len < 0 ? 0 : cap - m;
      }
      plan->len[b] = (int)len;
      if (m) {
        n = p.c.heads * ta_blocks(m * p.group, p.block);
        inc = (long long)n * ((len + m + (1 << TA_UNIT_SHIFT) - 1) >> TA_UNIT_SHIFT) * ta_cost(p, m);
      }
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, off);
      const int more = __shfl_up_sync(0xffffffffu, n, off);
      if (lane >= off) inc += up, n += more;
    }
    if (b < map.B) {
      plan->pre[b + 1] = run + inc;
      plan->items[b + 1] = items + n;
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
    items += __shfl_sync(0xffffffffu, n, 31);
  }
  const int begin = run >= 4ll * p.cost[0] * p.grid ? p.begin_cost : 0;
  for (int b = lane; b < map.B; b += 32) plan->pre[b + 1] += (long long)begin * plan->items[b + 1];   // its own entries
  if (lane == 0) {
    plan->pre[0] = 0;
    plan->begin = begin;
  }
}

// a / b for 0 <= a, 0 < b, in 32 bits where they fit (a 64-bit division takes hundreds of cycles).
__device__ __forceinline__ long long ta_div(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// Of an item whose cost counts from a0 on and that has nt units: the units before position x of the count.
__device__ __forceinline__ int ta_units_before(long long x, long long a0, int nt, int cost, int begin) {
  const long long n = x - a0 - begin;
  if (n <= 0) return 0;
  return n < (long long)nt * cost ? (int)((unsigned)n / (unsigned)cost) : nt;
}

// A run of units of one item in one CTA.
struct TaSeg {
  int b, h, rb, m, row0, rows;   // request, key head, row block; drafted rows, first row, rows of the block
  int tile0, n, nt, len, total;  // first unit, units, the item's units; committed and all tokens
  long long next;                // where the count goes on
  bool first;                    // of the item that the CTA's share begins in
};
__device__ __forceinline__ TaSeg ta_segment(const TreeAttnParams& p, const TaPlan& plan, long long u, long long u0, long long u1) {
  int lo = 0, hi = p.map.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (plan.pre[mid] <= u) lo = mid; else hi = mid;
  }
  TaSeg s;
  s.b = lo;                      // pre[lo] <= u < pre[lo + 1]: a request with units (the last of equal prefixes)
  s.row0 = p.map.offs[lo];
  s.m = p.map.offs[lo + 1] - s.row0;
  s.len = plan.len[lo];
  s.total = s.len + s.m;
  s.nt = (s.total + (1 << TA_UNIT_SHIFT) - 1) >> TA_UNIT_SHIFT;
  const int cost = ta_cost(p, s.m);
  const long long count = (long long)s.nt * cost + plan.begin, local = u - plan.pre[lo];
  const int item = (int)ta_div(local, count);
  const long long a0 = plan.pre[lo] + (long long)item * count;
  const int nrb = ta_blocks(s.m * p.group, p.block);
  s.h = item / nrb;
  s.rb = item - s.h * nrb;
  const int left = s.m * p.group - s.rb * p.block;
  s.rows = left < p.block ? left : p.block;
  s.next = a0 + count < u1 ? a0 + count : u1;
  s.tile0 = ta_units_before(u, a0, s.nt, cost, plan.begin);
  s.n = ta_units_before(s.next, a0, s.nt, cost, plan.begin) - s.tile0;
  s.first = u == u0;
  return s;
}
// The CTA's next run that has units, from position u on; false: there is none.
__device__ __forceinline__ bool ta_next(const TreeAttnParams& p, const TaPlan& plan, long long* u, long long u0, long long u1, TaSeg* s) {
  while (*u < u1) {
    *s = ta_segment(p, plan, *u, u0, u1);
    *u = s->next;
    if (s->n > 0) return true;
  }
  return false;
}

// A CTA's share of the count, from u0 to u1, and its first run.
struct TaShare {
  long long u0, u1, u;
  TaSeg s;
  bool more;
};
// By the whole CTA, up to and past its wait for the kernels before.  Lengths may be those kernels' results, but the same
// instructions are run once before the wait, on lengths of zero: they are in the caches when it counts.  (A first run of the
// planning takes 2.5 us; with the dry run before it one row over 2048 tokens takes 9.4 us against 10.3.)
__device__ __forceinline__ TaShare ta_begin(const TreeAttnParams& p, TaPlan* plan) {
  TaShare x;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (pass) {
      __syncthreads();         // the dry run's plan has been read
      pdl_wait();
      pdl_trigger();           // after the wait: the join may then read what this kernel's predecessors wrote before its own
    }
    if (threadIdx.x < 32) ta_plan(p, plan, pass, pass && blockIdx.x == 0);
    __syncthreads();
    const long long units = plan->pre[p.map.B], per = ta_div(units + p.grid - 1, p.grid);
    x.u0 = x.u = blockIdx.x * per;
    x.u1 = x.u0 + per < units ? x.u0 + per : units;
    x.more = ta_next(p, *plan, &x.u, x.u0, x.u1, &x.s);
  }
  return x;
}

// r / p.group for a row of a block: r < 64 p.group + 128, so the product is below 2^28 and the quotient off by less than
// r / 2^20 < 1 / p.group.
__device__ __forceinline__ int ta_by_group(const TreeAttnParams& p, int r) { return (int)(((uint32_t)r * p.per_group) >> 20); }

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
// Over codes a row of q enters the products as fp16 times 2^e, its largest magnitude mx at 2^14 to 2^15 (less for a subnormal
// mx, exactly all the same): e for any finite mx, and for infinity one with which finite elements stay finite.
__device__ __forceinline__ int ta_query_exponent(float mx) {
  const int e = 141 - (int)(__float_as_uint(mx) >> 23);
  return mx > 0.f ? (e < 126 ? e : 126) : 0;
}
// score -> exponent of 2, from products of a row times 2^e.  2^-e times the scale comes first: the scale alone may be subnormal.
__device__ __forceinline__ float ta_score_factor(float scale, int e) {
  return fminf(fabsf(scale) * pow2_exact(-e) * 1.4426950408889634f, 3.402823466e38f);
}
__device__ __forceinline__ bool ta_half_bad(uint32_t h) { return (h & 0x7c00u) == 0x7c00u; }

// Where a CTA's run of an item leaves its partial sums.
__device__ __forceinline__ size_t ta_slot(const TaSeg& s) { return 2 * (size_t)blockIdx.x + (s.first ? 0 : 1); }

cudaError_t launch_tree_attn_wide(const TreeAttnParams& p, cudaStream_t s);     // blocks of 128 rows
cudaError_t launch_tree_attn_narrow(const TreeAttnParams& p, cudaStream_t s);   // of 16 or 32

}  // namespace sv
