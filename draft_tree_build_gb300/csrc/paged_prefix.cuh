// What the two launches of shared-prefix attention share.
#pragma once

#include "paged.cuh"
#include "paged_units.cuh"

namespace bastion {

// Own slots in tables of at most this many slots go to paged_prefix_own.cu, others to
// the one-token kernel.  By the table's width, as the lengths are known on the GPU alone: a table
// much wider than its requests loses what short slots gain (tables of 4,096 slots for 33, 512, 257 and
// 64: 4 requests 11.8 -> 14.0 us, 64 55 -> 55, 61 of 64-element heads 22.3 -> 28.4, 256 163 -> 180).  Whole calls behind 2,000 shared tokens, 32/8 heads, one way
// and the other: D = 64: 500 slots, 1, 8, 64, 200 requests: 14.4 and 16.3 us, 19.6 and 23.7,
// 29.4 and 38.2, 62.7 and 71.1; 1,000 slots 19.1 and 19.1, 24.2 and 24.6, 41.1 and 50.1, 99 and 123;
// 2,000 slots 27.9 and 20.0, 32.8 and 29.3, 64 and 80, 170 and 222 (few requests lose where many gain; the limit is
// where a single one no longer gains).  D = 128, whose outputs take
// twice the registers, so that half as many warps are on an SM: 64 slots, 8 requests 17.0
// and 21.7, 256 53.0 and 58.0; 128 slots 23.5 and 21.9, 70.5 and 60.0.
__host__ __device__ constexpr int own_slots(int D) { return D == 64 ? 1024 : 64; }

// Where the join finds the parts of a request's rows of one KV head.  Part p is of
// CTA x = p / planes, plane p % planes: at place0 + plane * step for x = 0 and at
// place1 + (x - 1) * 512 + plane * step for the others (a CTA has two slots of two
// planes of 128 rows).
struct alignas(16) PartsRec {
  int32_t parts, two;  // how many, and whether of two planes
  int32_t place0, place1, step;
  int32_t whole;       // in rows, not in parts
  int32_t rows, first; // rows of the M tile and the request's first among them
};

struct PrefixArgs {
  const int32_t *table, *len, *start;  // the groups' prefixes
  int n_groups, max_pages, cap;
  int Hq, G, nb;  // nb = 128 / G requests an M tile
  float scale_log2;
  int swap;
  PartsRec *rec;   // [B, Hkv]
  float *own;      // [B, Hq, D], normalised
  float *own_lse;  // [B, Hq], base 2
  float *rows;     // [2][B, Hq, D]: units of one CTA
  float2 *rows_ml;
  float *parts;    // [2 kMaxParts][2][128][D]: units of several
  float2 *parts_ml;
  int n_ctas;
  const uint16_t *q;
  int64_t q_st_b;
  const int32_t *seq_len;
  uint16_t *out;
  float *lse;
  int32_t *status;
};

// --------------------------------------------------------------------------- parts

// An M tile's part is its R rows, four elements of each side by side: element d of
// row i at place * D + (d / 4 * R + i) * 4 + d % 4, so that a warp of rows writes,
// and the join reads, whole sectors; reference and sum at place + i.
__device__ __forceinline__ size_t whole_part(int plane, int head, int req, const Paged &c, int G) {
  return (((size_t)plane * c.Hkv + head) * c.B + req) * G;
}
__device__ __forceinline__ size_t cut_part(int slot, int plane) { return ((size_t)slot * 2 + plane) * 128; }

cudaError_t launch_prefix_own(bool half, int sms, const Paged &c, const PrefixArgs &a, cudaStream_t stream);
cudaError_t launch_prefix_join(bool half, int sms, const Paged &c, const PrefixArgs &a, cudaStream_t stream);

}  // namespace bastion
