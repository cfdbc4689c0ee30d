// Attention of a group's rows over the prefix that its requests share: parameters, and how the work is dealt.
//
// Every (group, key head, block of up to 256 rows) is an item of tiles of 128 tokens.  The items, in order, are dealt to the CTAs in
// equal contiguous shares of their cost, all of it known on the host.  Each run of an item in a CTA leaves fp32 sums (with their
// maximum and weight) in the workspace, at the place item + CTA: neither goes down from run to run, and one of them goes up.
#pragma once

#include "tree_attn.cuh"

namespace sv {

constexpr int PX_ROWS = 256;          // rows per block: two matrices of 128 lanes

struct PrefixParams {
  CUtensorMap tk, tv;                 // 16-bit caches, as in tree attention
  KvCache c;
  const int32_t* table;
  int table_pages;
  const __nv_bfloat16* q; int ldq;
  int heads_per;                      // query heads per key head
  float scale;
  float* partial;                     // [items + grid][256][dim]
  float* stats;                       // [items + grid][2][256]: maximum (as an exponent of 2) and weight
  int grid, n;                        // CTAs; groups with a prefix
  int cost[2], begin_cost;            // of a tile of a block with up to 128 rows, and with more; of beginning an item
  long long per;                      // a CTA's share
  long long pre[MAX_BATCH + 1];       // cost of the groups before
  int items[MAX_BATCH + 1];           // their items
  int row0[MAX_BATCH], rows[MAX_BATCH];       // first row; rows times heads_per
  int tokens[MAX_BATCH], request[MAX_BATCH];  // of the prefix; the request whose pages are read
  short group[MAX_BATCH];             // of each request: its place among these groups, or -1
};

// The blocks of a group: all but the last have 256 rows.
struct PxGroup {
  int blocks, last, nt;               // blocks; whether the last has more than 128 rows; tiles
  long long full, tail, span;         // cost of a block, of the last, of a key head
};
__host__ __device__ __forceinline__ PxGroup px_group(const PrefixParams& p, int rows, int tokens) {
  PxGroup g;
  g.blocks = (rows + PX_ROWS - 1) / PX_ROWS;
  g.last = rows - (g.blocks - 1) * PX_ROWS > PX_ROWS / 2;
  g.nt = (tokens + 127) / 128;
  g.full = (long long)g.nt * p.cost[1] + p.begin_cost;
  g.tail = (long long)g.nt * p.cost[g.last] + p.begin_cost;
  g.span = (g.blocks - 1) * g.full + g.tail;
  return g;
}

cudaError_t launch_tree_attn_prefix(const PrefixParams& p, cudaStream_t s);

}  // namespace sv
