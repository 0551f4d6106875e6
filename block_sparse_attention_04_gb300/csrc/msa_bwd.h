// The attention's backward pass: what its kernels share (internal interface).
//
// Row statistics.  The kernels recompute P = 2^(s scale log2e - lse log2e) and
// dS = P (dP - delta); the two numbers of a (query, head) row are kept in groups of
// 8 rows, 128 bytes: [8 rows][8 bf16], -lse / scale in three parts at 0..2 and -delta
// alike at 4..6, zeros at 3 and 7: products with ones add them to S and dP.
// (-lse log2e where scale log2e is below 2^-100 and scores count for nothing.)
//   dense    group ((b H + h) ngroups + i/8), a tile's 16 groups in a row; rows past
//            the last query hold -16384 (times 1 / scale log2e) and 0: their P and dS
//            vanish.  Next to it, for dQ's CTAs, 64 bytes a group: eight
//            -lse log2e, then eight -delta.
//   sparse   group (((b T + i) G + g) rpe/8 + head/8): an entry's rows; heads past
//            the group's last as above, and one such group behind all others
#pragma once
#include "msa_train.h"

namespace msa {

constexpr int kStatBytes = 64;          // a group of 8 rows as numbers
constexpr int kAugBytes = 128;          // ... as operands
constexpr int kBwdSms = 152;            // what sizes of scratch are made for
constexpr int kChunkRows = 64;          // query rows whose list entries keep their order

// A unit is a piece of the work of one KV block: x = kb | g << 15 | b << 18; dense: y =
// first tile, z = tiles (a head's query tiles are consecutive); sparse: y = first entry (a
// multiple of R), z = entries; w = slot of the piece's partial sums, or -1 where it is the
// block's only one.  A list's entries start at a multiple of R, so that entry e is in tile
// e / R of the pass.
//
// Layouts of partial sums, in which a warp's 32-byte stores are contiguous:
//   part_dq  [tile][D/16][128 rows][16 dims] bf16     row (e % R) rpe + head of the group
//   part_kv  [slot][dv, dk][D/8][128 tokens][8 dims] fp32
struct BwdArgs {
  Shape s;
  Positions pos;
  int t0, Tp;                // queries of the pass: [t0, t0 + Tp) of every sequence
  int nbl;                   // KV blocks per sequence in the item space
  int hpg, rpe, R;           // heads per group; sparse: rows per entry, entries per tile
  int nqt;                   // dense: 128-query tiles per sequence
  int piece;                 // tiles per unit (at most)
  const int32_t* sel;        // sparse: the selection
  int32_t* cnt;              // [B][chunks][G][nbl]: entries per chunk, then those before
  int chunks;
  int32_t* count;            // [G][B][nbl] entries of a list
  int32_t* off;              // [G][B][nbl] its first entry
  int32_t* entries;          // (i - t0) * 16 + slot
  int32_t* where;            // [B*Tp][G][16]: the entry of each selected id, -1: none
  int4* units;
  int* n_units;              // [2]: units, partial slots
  int4* slots;               // per slot: (b, g, kb packed as x; its unit's slots, 0 but for the first)
  int max_slots;
  int* next_unit;            // counter of taken units
  const uint8_t* stat;       // as operands
  uint32_t stat_groups;      // dense: groups per (b, h); sparse: index of the neutral group
  bool no_scores;            // scale log2e below 2^-100
  uint16_t* part_dq;         // sparse: dq of each tile, without the scale
  float* part_kv;            // dv, dk of each slot (dk without the scale)
  float* acc;                // several passes: running dv, dk [2][B][max_blocks][128][G][D]
  bool first, last;          // pass
  uint16_t *dq, *dk, *dv;
  int* status;
  // poll caps of the pipeline waits, KV-outer and dQ's (0: wall-clock bound only)
  uint32_t wait_polls, q_wait_polls;
  // tests of waits that run out: the copy of a KV-outer CTA, of a dQ CTA that is late
  // (-1: none), and by how much
  int late_kv, late_q;
  uint32_t late_ns;
  // dense: dQ by (query tile, head) items x splits of their key blocks
  int kv_ctas;               // CTAs of the launch that work on units; those behind take items
  int q_items, q_splits;
  int* next_item;            // counter of taken items
  const uint8_t* nums;       // statistics as numbers
  const uint16_t* q;
  float* part_q;             // q_splits > 1: [items][splits][128][D] partial dq
};

// Dense: the first query tile that sees block kb of sequence b (nqt: none does).
__host__ __device__ inline int bwd_first_tile(const BwdArgs& a, int b, int kb) {
  const int64_t i0 = (int64_t)kb * kBlock - a.pos.q_start[b];
  if (i0 >= a.s.T) return a.nqt;
  return i0 > 0 ? (int)(i0 / 128) : 0;
}

// Whether scores are scaled to nothing.
inline bool bwd_no_scores(const Shape& s) {
  const float sl = s.scale * 1.4426950408889634f;
  return (sl < 0 ? -sl : sl) < 0x1p-100f;
}

// Preparation: row statistics (stat: dense only; aug: as operands; clears *status), lists (sparse), units.
cudaError_t launch_bwd_stats(const Shape& s, const Positions& pos, const AttnBwd& a, int rpe,
                             uint8_t* stat, uint8_t* aug, uint32_t stat_groups, int* status,
                             cudaStream_t st);
cudaError_t launch_bwd_lists(const BwdArgs& a, cudaStream_t st);
cudaError_t launch_bwd_units(const BwdArgs& a, cudaStream_t st);
// dK and dV, one owner per KV block; sparse: dQ's parts, dense: dQ.
cudaError_t launch_bwd_kv(const BwdArgs& a, const AttnBwd& t, cudaStream_t st);
// Joins: dQ from the selected blocks' parts; dK and dV of blocks in several pieces.
cudaError_t launch_bwd_join_q(const BwdArgs& a, cudaStream_t st);
cudaError_t launch_bwd_join_kv(const BwdArgs& a, cudaStream_t st);

}  // namespace msa
