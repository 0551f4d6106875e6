// The attention's backward pass (msa_sparse_attn_bwd, msa_dense_attn_bwd): its scratch
// and the sequence of its kernels.
//   dense    statistics; units; dK and dV (KV-outer) and dQ (query-outer) in one launch
//   sparse   statistics; per pass of at most 8192 query rows: lists, units; dK, dV and
//            dQ's parts (KV-outer); the parts' sums.  Several passes add dK and dV up
//            in fp32.
// Dense takes two passes of four and three products where one of five would do: dQ
// would then need one sum per (query, head) over all key blocks, i.e. atomic adds (whose
// order changes the bits) of 128 x D fp32 per tile.
#include "msa_bwd.h"
#include "msa_tc.h"
#include "msa_tma.h"

namespace msa {
namespace {

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// Tiles per unit: a block's work is divided where it would hold up the others (the largest
// units go first): sparse, where it is more than a quarter of a CTA's share of all `tiles`
// (most of the tiles there might be; 8192 queries at 48/8 heads: the KV-outer kernel 1005 us,
// 1131 with two thirds, 976 with an eighth, whose joins take that back; 2048 of 32K 336,
// 339, 357).  Dense, two thirds: the tiles are known and the sizes go down evenly
// (4 x 2048 tokens 642 us in all, 665 with a quarter).  Not below 16 tiles: a piece costs
// about three tiles' time, K and V, the sums' way out and back.  A divided block of
// n > piece tiles has ceil(n / piece) <= 2 n / piece slots, so a call has at most
// 2 tiles / piece, and no call of up to `tiles` tiles more than the second bound.
constexpr int kMinPiece = 16;
int piece_tiles(int64_t tiles, bool sparse) {
  const int64_t p = (sparse ? tiles / (4 * kBwdSms) : tiles * 2 / (3 * kBwdSms)) + 1;
  return (int)(p < kMinPiece ? kMinPiece : (p > (1 << 28) ? 1 << 28 : p));
}
int sparse_slots(int64_t tiles) { return (int)(2 * tiles / piece_tiles(tiles, true)); }
int most_slots(int64_t tiles) {
  const int64_t n = 2 * tiles / kMinPiece;
  return (int)(n < 8 * kBwdSms ? n : 8 * kBwdSms);
}

int rows_per_entry(const Shape& s) { return s.H / s.G <= 8 ? 8 : 16; }

// Tiles of a dense call, or with `piece` the slots of its divided blocks.
int64_t dense_tiles(const BwdArgs& a, int piece = 0) {
  int64_t n = 0;
  auto add = [&](int64_t blocks, int query_tiles) {
    const int64_t t = (int64_t)query_tiles * a.hpg;
    n += blocks * a.s.G * (piece == 0 ? t : (t > piece ? (t + piece - 1) / piece : 0));
  };
  for (int b = 0; b < a.s.B; ++b) {
    // blocks up to the first query's see every tile, later ones fewer
    const int first = a.pos.q_start[b] / kBlock;
    const int last = (int)(((int64_t)a.pos.q_start[b] + a.s.T - 1) / kBlock);
    add(first + 1, a.nqt);
    for (int kb = first + 1; kb <= last; ++kb) add(1, a.nqt - bwd_first_tile(a, b, kb));
  }
  return n;
}

// Tiles of a call or a pass, at most.
int64_t max_tiles(const Shape& s, bool sparse, int tp, int nbl) {
  const int64_t lists = (int64_t)s.B * nbl * s.G;
  if (sparse) {
    const int64_t entries = (int64_t)s.B * tp * s.G * kTopk, r = 128 / rows_per_entry(s);
    return entries / r + (lists < entries ? lists : entries);
  }
  return lists * (s.H / s.G) * ((s.T + 127) / 128);
}

// Dense: at most this many (item, split) partials.
constexpr int kMaxQParts = 4 * kBwdSms;
int q_items(const Shape& s) { return (s.T + 127) / 128 * s.B * s.H; }

struct Layout {
  size_t stat, aug, cnt, count, off, entries, where, units, slots, part_dq, part_kv, acc, part_q, total;
  uint32_t stat_groups;
  int chunks;
};

Layout layout(const Shape& s, bool sparse) {
  Layout L{};
  const int tp = pass_len(s), nbl = s.max_blocks;
  const int64_t lists = (int64_t)s.B * nbl * s.G;
  const int rpe = rows_per_entry(s);
  size_t o = 256;                        // the counters
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  const int64_t tiles = max_tiles(s, sparse, tp, nbl);
  const int slots = most_slots(tiles);
  if (sparse) {
    L.stat_groups = (uint32_t)((size_t)s.B * s.T * s.G * (rpe / 8));
    L.aug = take(((size_t)L.stat_groups + 1) * kAugBytes);
    L.chunks = (tp + kChunkRows - 1) / kChunkRows;
    L.cnt = take((size_t)s.B * L.chunks * s.G * nbl * sizeof(int32_t));
    L.count = take(lists * sizeof(int32_t));
    L.off = take(lists * sizeof(int32_t));
    L.entries = take((size_t)tiles * (128 / rpe) * sizeof(int32_t));
    L.where = take((size_t)s.B * tp * s.G * kTopk * sizeof(int32_t));
    L.part_dq = take((size_t)tiles * 128 * s.D * 2);
    if (tp < s.T) L.acc = take((size_t)lists * kBlock * s.D * 2 * sizeof(float));
  } else {
    L.stat_groups = (uint32_t)((s.T + 127) / 128 * 16);
    L.stat = take((size_t)s.B * s.H * L.stat_groups * kStatBytes);
    L.aug = take((size_t)s.B * s.H * L.stat_groups * kAugBytes);
    const int items = q_items(s);
    if (items < kMaxQParts) L.part_q = take((size_t)kMaxQParts * 128 * s.D * sizeof(float));
  }
  L.units = take((lists + slots) * sizeof(int4));
  L.slots = take((size_t)slots * sizeof(int4));
  L.part_kv = take((size_t)slots * 2 * kBlock * s.D * sizeof(float));
  L.total = o;
  return L;
}

// Few items: the key blocks of each over several CTAs, at least 4 blocks a split.
int dense_q_splits(const BwdArgs& a) {
  if (a.q_items >= kMaxQParts) return 1;
  int blocks = 1;
  for (int b = 0; b < a.s.B; ++b) {
    const int n = (int)(((int64_t)a.pos.q_start[b] + a.s.T - 1) / kBlock) + 1;
    blocks = n > blocks ? n : blocks;
  }
  const int by_parts = kMaxQParts / a.q_items, by_blocks = blocks / 4;
  const int n = by_parts < by_blocks ? by_parts : by_blocks;
  return n < 1 ? 1 : n;
}

}  // namespace

size_t attn_bwd_scratch_bytes(const Shape& s, bool sparse) { return layout(s, sparse).total; }

cudaError_t launch_attn_bwd(const Shape& s, const Positions& pos, const AttnBwd& t, int* status,
                            char* base, cudaStream_t st) {
  const bool sparse = t.sel != nullptr;
  const Layout L = layout(s, sparse);
  BwdArgs a{};
  a.s = s;
  a.pos = pos;
  a.hpg = s.H / s.G;
  a.rpe = rows_per_entry(s);
  a.R = 128 / a.rpe;
  a.nqt = (s.T + 127) / 128;
  a.sel = t.sel;
  a.n_units = reinterpret_cast<int*>(base);
  a.next_unit = a.n_units + 2;
  a.next_item = a.n_units + 3;
  uint8_t* const stat = sparse ? nullptr : reinterpret_cast<uint8_t*>(base + L.stat);
  uint8_t* const aug = reinterpret_cast<uint8_t*>(base + L.aug);
  a.stat = aug;
  a.no_scores = bwd_no_scores(s);
  a.stat_groups = L.stat_groups;
  a.chunks = L.chunks;
  a.cnt = reinterpret_cast<int32_t*>(base + L.cnt);
  a.count = reinterpret_cast<int32_t*>(base + L.count);
  a.off = reinterpret_cast<int32_t*>(base + L.off);
  a.entries = reinterpret_cast<int32_t*>(base + L.entries);
  a.where = reinterpret_cast<int32_t*>(base + L.where);
  a.units = reinterpret_cast<int4*>(base + L.units);
  a.slots = reinterpret_cast<int4*>(base + L.slots);
  a.part_dq = reinterpret_cast<uint16_t*>(base + L.part_dq);
  a.part_kv = reinterpret_cast<float*>(base + L.part_kv);
  a.acc = reinterpret_cast<float*>(base + L.acc);
  a.dq = t.dq;
  a.dk = t.dk;
  a.dv = t.dv;
  a.status = status;
  const CopyDelay delay = debug_copy_delay();
  a.late_kv = delay.kind == MSA_DEBUG_BWD_KV ? delay.at : -1;
  a.late_q = delay.kind == MSA_DEBUG_BWD_DQ ? delay.at : -1;
  a.late_ns = delay.ns;
  a.wait_polls = delay.kind == MSA_DEBUG_BWD_DQ ? 0 : debug_wait_polls();
  a.q_wait_polls = delay.kind == MSA_DEBUG_BWD_KV ? 0 : debug_wait_polls();
  if (!sparse) {
    a.q_items = q_items(s);
    a.q_splits = dense_q_splits(a);
    a.nums = stat;
    a.q = t.q;
    a.part_q = reinterpret_cast<float*>(base + L.part_q);
  }
  int max_len = 1;
  for (int b = 0; b < s.B; ++b) max_len = pos.kv_len[b] > max_len ? pos.kv_len[b] : max_len;
  a.nbl = (max_len + kBlock - 1) / kBlock;
  cudaError_t e;
  if ((e = launch_bwd_stats(s, pos, t, sparse ? a.rpe : 0, stat, aug, L.stat_groups, status,
                            st)) !=
      cudaSuccess)
    return e;
  const int tp = sparse ? pass_len(s) : s.T;
  for (int t0 = 0; t0 < s.T; t0 += tp) {
    a.t0 = t0;
    a.Tp = tp < s.T - t0 ? tp : s.T - t0;
    a.first = t0 == 0;
    a.last = t0 + tp >= s.T;
    const int64_t tiles = sparse ? max_tiles(s, true, a.Tp, a.nbl) : dense_tiles(a);
    a.piece = piece_tiles(tiles, sparse);
    a.max_slots = sparse ? sparse_slots(tiles) : (int)dense_tiles(a, a.piece);
    if ((e = sparse ? launch_bwd_lists(a, st) : launch_bwd_units(a, st)) != cudaSuccess) return e;
    if ((e = launch_bwd_kv(a, t, st)) != cudaSuccess) return e;
    if ((e = launch_bwd_join_kv(a, st)) != cudaSuccess) return e;
    if (sparse && (e = launch_bwd_join_q(a, st)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace msa
