// How a prefill call's work is cut into the CTAs' shares.
//
// A unit is a (sequence, KV head, row tile): up to 256 query rows (a row is one query
// token and one of the G query heads of the KV head; whole tokens, token-major) against
// the positions its last token sees. Units lie on a line in the order sequence, KV head,
// tile; a unit is kPfUnitCost positions (its query load and output) plus the positions its
// last row sees. Every CTA takes an equal stretch of the line; tile k of a unit (positions
// 128k .. 128k + 127) belongs to the CTA whose stretch holds its first position. A unit
// cut by a stretch's end becomes pieces that are merged by the last to finish. While stretches
// are short (kPfWholeShare) a unit of at most kPfWhole positions is not cut: all of it belongs
// to the CTA whose stretch holds its start, since writing and merging pieces takes as long as some
// five tiles (eight prompts of 512 tokens: 43 us; 49 with kPfWholeShare 1600, where they are cut). One
// bf16 prompt of 32 + 8 heads, whole / cut: 512 tokens 17.1 / 20.9 us, 1024 25.2 / 31.2, 1536 41.1 / 37.1, 2048
// (a share of 2425, so cut) 49.0 / 47.2.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pkv_internal.h"
#include "prefill_row.cuh"

namespace pkv {

constexpr int kPfRows = 256;          // query rows of a unit: two tiles of the MMA's M
constexpr int kPfTile = 128;          // positions of a KV tile
// A unit's fixed cost, in positions (256 / 320 / 384 gave an 8192-token bf16 prompt 372 / 370 /
// 360 us; 512 no less).
constexpr int kPfUnitCost = 384;
// Of a sequence whose unit fills one row tile at most (single decode rows): its tiles and outputs
// take less. (With the same cost a chunk's CTAs end at 109 us, those of 31 decode rows beside it at
// 88. 0 / 128 / 256 / 384 gave that batch 133 / 117 / 118 / 120 us, two chunks of 512 and 30 decode
// rows over INT8 139 / 124 / 130 / 131.)
constexpr int kPfUnitCostFew = 128;
__device__ __forceinline__ int pf_unit_cost(int n, int group) {
  return n * group <= 128 ? kPfUnitCostFew : kPfUnitCost;   // (n < 2^31 / num_q_heads)
}
constexpr int kPfWhole = 8 * kPfTile, kPfWholeShare = 2400;
// A unit of more pieces is joined in groups first: one CTA that adds up 19 pieces of two full row
// tiles takes 30 us at the call's end (64 tokens over 131008: 141 us against 122; 4 to 9 alike).
constexpr int kPfJoin = 6;
constexpr int kPfMinShare = 3 * kPfTile + kPfUnitCost;   // where units are cut: at least one whole tile a piece

// Tokens of one TMA box of query rows, and of a unit (whole boxes). Boxes start on the
// swizzle's 8-row atoms, 32 rows or the next possible number each, so that a short unit
// copies little; where such boxes leave more than a quarter of the rows empty (a large
// odd group), one box of as many tokens as fit.
struct PfBox {
  int tokens, unit;
};
inline PfBox pf_box(int group) {
  int atom = 1;
  while (atom * group % 8 != 0) ++atom;
  int bt = atom;
  while ((bt + atom) * group <= 32) bt += atom;
  const int most = kPfRows / group, unit = most / bt * bt;
  if (4 * unit < 3 * most) return {most, most};
  return {bt, unit};
}

// Shared description of a CTA's stretch, written by pf_plan.
struct PfStart {
  long long b0, b1, share, ub;
  int s, h, t, any;
};

// A place on the walk: the current unit and its sequence.
struct PfPos {
  long long ub;              // line position of the unit
  int s, h, t;
  int n, qb, ctx;            // of sequence s
};

struct PfWalk {
  const PrefillArgs& a;
  const PfStart& st;
  PfPos p;

  __device__ PfWalk(const PrefillArgs& args, const PfStart& start) : a(args), st(start) {
    p.ub = st.ub;
    p.s = st.s;
    p.h = st.h;
    p.t = st.t;
    load();
  }
  __device__ void load() {
    const PrefillSeq q = prefill_seq(a, p.s);
    p.n = q.n;
    p.qb = q.qb;
    p.ctx = q.ctx;
  }
  __device__ bool done() const { return p.ub >= st.b1; }
  __device__ int past() const { return p.ctx - p.n; }
  __device__ int pastp() const { return max(past(), 0); }
  __device__ int len() const { return pastp() + min((p.t + 1) * a.unit_tokens, p.n); }
  __device__ int cost() const { return pf_unit_cost(p.n, a.group); }
  __device__ void advance() {
    p.ub += cost() + len();
    if (++p.t * a.unit_tokens < p.n) return;
    p.t = 0;
    if (++p.h < a.num_kv_heads) return;
    p.h = 0;
    if (p.ub >= st.b1) return;
    do {
      ++p.s;
      load();
    } while (p.n == 0);   // ub < b1 <= the line's end: another sequence with rows follows
  }
  __device__ int owner(int k) const {
    return static_cast<int>((p.ub + cost() + static_cast<long long>(kPfTile) * k) / st.share);
  }
};

// This CTA's piece of a unit, as one warp works it out and the others read it from shared
// memory: the walk's 64-bit arithmetic, run by every role, was a good part of the kernel's code,
// and what runs once a piece finds its code evicted by the loops.
struct PfPiece {
  int end;                   // no further piece
  int s, h;                  // sequence, KV head
  int qb, past, ctx;         // first query row, positions before the first query token (may be < 0), context
  int j0, rows;              // first query token of the unit, its rows
  int ka, klast;             // KV tiles [ka, klast) ...
  int kb[2];                 // ... of which row tile i takes those below kb[i] (none: kb <= ka)
  int rot;                   // the tiles are taken from ka + rot on, then those from ka: step k takes tile at(k)
  int tail;                  // the step whose tile's V rows end behind the context inside a block, else -1

  __device__ static int at(int k, int rot, int ka, int klast) {
    const int t = k + rot;
    return t < klast ? t : t - (klast - ka);
  }
  int first[2], pieces[2];   // of a row tile cut by a stretch's end: its first CTA, its pieces (1: not cut)
};

// False if the CTA has no tile of the unit.
__device__ inline bool pf_piece(const PfWalk& w, volatile PfPiece* to) {
  const int G = w.a.group, qt = w.a.unit_tokens;
  const int j0 = w.p.t * qt, rows = min(qt, w.p.n - j0) * G;
  const int k_all = (w.len() + kPfTile - 1) / kPfTile;
  const long long x0 = w.st.b0 - w.p.ub - w.cost(), x1 = w.st.b1 - w.p.ub - w.cost();
  int ka = x0 <= 0 ? 0 : static_cast<int>((x0 + kPfTile - 1) / kPfTile);
  int kx = x1 <= 0 ? 0 : static_cast<int>(min((x1 + kPfTile - 1) / kPfTile, static_cast<long long>(k_all)));
  if (w.len() <= kPfWhole && w.st.share < kPfWholeShare) {
    ka = 0;
    kx = w.p.ub >= w.st.b0 ? k_all : 0;   // (the walk passes no unit that starts behind the stretch)
  }
  int kend[2] = {k_all, 0};   // tiles of the whole unit row tile i needs
  if (rows > 128) {
    kend[0] = (w.pastp() + j0 + 127 / G + 1 + kPfTile - 1) / kPfTile;
    kend[1] = k_all;
  }
  const int klast = min(kx, k_all);
  if (ka >= klast) return false;
  to->end = 0;
  to->s = w.p.s;
  to->h = w.p.h;
  to->qb = w.p.qb;
  to->past = w.past();
  to->ctx = w.p.ctx;
  to->j0 = j0;
  to->rows = rows;
  to->ka = ka;
  to->klast = klast;
  // Several units of one head read the same tiles. So that they do so at about the same time, out
  // of L2, the CTA begins a cut unit with the tile whose line length is its own elapsed one,
  // modulo a stretch's (128 tokens over 130944: 204 us in rising order, where each unit reads the
  // context from memory, against 194; of whole units too, a ragged E5M2 batch lost 9 %). Not
  // where one row tile takes fewer of the tiles than the other.
  int rot = 0;
  bool level = w.p.n > qt && (ka > 0 || kx < k_all);
  for (int i = 0; i < 2; ++i) level &= min(kx, kend[i]) <= ka || kend[i] >= klast;
  if (level) {
    const long long e0 = static_cast<long long>(kPfTile) * ka - x0;   // elapsed at the piece's start
    const long long m = x0 > 0 ? (x0 + w.st.share - 1) / w.st.share : 0;
    const long long k0 = (e0 + m * w.st.share + kPfTile - 1) / kPfTile;
    if (k0 > ka && k0 < klast) rot = static_cast<int>(k0) - ka;
  }
  to->rot = rot;
  int tail = w.p.ctx & 15 ? w.p.ctx / kPfTile : -1;
  if (tail >= ka && tail < klast) tail = tail - rot < ka ? tail - rot + klast - ka : tail - rot;
  else tail = -1;
  to->tail = tail;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    to->kb[i] = min(kx, kend[i]);
    const bool whole = ka == 0 && kx >= kend[i];
    const int first = whole || kend[i] == 0 ? 0 : w.owner(0);
    to->first[i] = first;
    to->pieces[i] = whole || kend[i] == 0 ? 1 : w.owner(kend[i] - 1) - first + 1;
  }
  return true;
}

// Line length of one KV head of a sequence: T units of cost + pastp + min((t+1) qt, n).
__device__ __forceinline__ long long pf_head_len(int n, int pastp, int qt, int group) {
  if (n == 0) return 0;
  const long long T = (n + qt - 1) / qt;
  return T * (pf_unit_cost(n, group) + pastp) + static_cast<long long>(qt) * ((T - 1) * T / 2) + n;
}

// The CTA's start on the line. Every thread of the CTA takes part; scratch: one long long a
// warp. CTA 0 flags the sequences that break a rule. Ends with a barrier.
__device__ inline void pf_plan(const PrefillArgs& a, long long* scratch, PfStart* st) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int per = (a.num_seqs + blockDim.x - 1) / blockDim.x;
  const int s0 = tid * per, s1 = min(s0 + per, a.num_seqs);
  if (tid == 0) st->any = 0;
  long long mine = 0;
  bool bad = false, cut = false;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    const PrefillSeq p = prefill_seq(a, s);
    bad |= p.bad;
    cut |= p.n > 0 && max(p.ctx, p.n) > kPfWhole;   // its longest unit
    mine += a.num_kv_heads * pf_head_len(p.n, max(p.past(), 0), a.unit_tokens, a.group);
  }
  if (bad && blockIdx.x == 0 && a.status) atomicOr(a.status, kDevBadCtx);
  long long incl = mine;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scratch[warp] = incl;
  cut = __syncthreads_or(cut);
  long long total = 0, excl = incl - mine;
#pragma unroll 1
  for (int w = 0; w < nw; ++w) {
    if (w < warp) excl += scratch[w];
    total += scratch[w];
  }
  long long share = (total + gridDim.x - 1) / gridDim.x;
  if (cut && share < kPfMinShare) share = kPfMinShare;
  const long long b0 = static_cast<long long>(blockIdx.x) * share;
  if (b0 < total && excl <= b0 && b0 < excl + mine) {
    long long at = excl;
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      const PrefillSeq p = prefill_seq(a, s);
      const int pastp = max(p.past(), 0), qt = a.unit_tokens;
      const long long head = pf_head_len(p.n, pastp, qt, a.group);
      if (b0 >= at + a.num_kv_heads * head) {
        at += a.num_kv_heads * head;
        continue;
      }
      const int h = static_cast<int>((b0 - at) / head);
      const long long rem = b0 - at - h * head;
      // the unit that holds position rem: units before t take t (cost + pastp) + qt t (t + 1) / 2
      const long long c = pf_unit_cost(p.n, a.group) + pastp;
      int lo = 0, hi = (p.n + qt - 1) / qt - 1;
#pragma unroll 1
      while (lo < hi) {
        const long long t = (lo + hi + 1) / 2;
        if (t * c + qt * (t * (t + 1) / 2) <= rem) lo = static_cast<int>(t);
        else hi = static_cast<int>(t) - 1;
      }
      st->b0 = b0;
      st->b1 = min(b0 + share, total);
      st->share = share;
      st->ub = at + h * head + lo * c + static_cast<long long>(qt) * (static_cast<long long>(lo) * (lo + 1) / 2);
      st->s = s;
      st->h = h;
      st->t = lo;
      st->any = 1;
      break;
    }
  }
  __syncthreads();
}

}  // namespace pkv
