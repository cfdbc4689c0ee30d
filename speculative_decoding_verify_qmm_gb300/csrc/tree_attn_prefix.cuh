// Attention of a group's rows over the prefix that its requests share: parameters, and how the work is dealt.
//
// Every (group, key head, block of up to 256 rows) is an item of tiles of 128 tokens, cut into equal pieces; a CTA takes some
// consecutive pieces whole, and those of one item among them as one run.  All of it is known on the host.  A run leaves fp32 sums (with
// their maximum and weight) in the workspace, at item plus CTA: neither goes down from run to run, and one of them goes up.  (So their
// number follows from the rows, whatever the pieces: a workspace for the largest batch does for all.)
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
  float* partial;                     // [items + CTAs][256][dim]
  float* stats;                       // [items + CTAs][256][8]: maximum (as an exponent of 2) and weight of a row, in a sector of its own
  int grid, n;                        // CTAs; groups with a prefix
  int pieces[MAX_BATCH + 1];          // of the groups before
  int items[MAX_BATCH];               // likewise
  int splits[MAX_BATCH];              // pieces of an item
  int row0[MAX_BATCH], rows[MAX_BATCH];       // first row; rows times heads_per
  int tokens[MAX_BATCH], request[MAX_BATCH];  // of the prefix; the request whose pages are read
  short group[MAX_BATCH];             // of each request: its place among these groups, or -1
};

__host__ __device__ __forceinline__ int px_blocks(int rows) { return (rows + PX_ROWS - 1) / PX_ROWS; }
__host__ __device__ __forceinline__ int px_tiles(int tokens) { return (tokens + 127) / 128; }
// The first piece of CTA c, and the CTA of a piece.
__host__ __device__ __forceinline__ int px_first(int all, int grid, int c) { return (int)((long long)c * all / grid); }
__host__ __device__ __forceinline__ int px_cta(int all, int grid, int piece) { return (int)((((long long)piece + 1) * grid - 1) / all); }
// Whether a block has more rows than one matrix.
__host__ __device__ __forceinline__ bool px_pair(int rows, int rb) { return rows - rb * PX_ROWS > PX_ROWS / 2; }

cudaError_t launch_tree_attn_prefix(const PrefixParams& p, cudaStream_t s);

}  // namespace sv
