// How the attention kernels share out their work.
//
// An item is `tokens` consecutive query tokens of one sequence with all the query heads of one
// key-value head: rows token * G + g, so a key tile that is loaded once serves every head that
// shares it. Its cost is the number of kTileKeys-key tiles that its last token sees, at least 1
// (an item that sees nothing still has to write zeros), and `extra`, the time that an item takes
// beside its tiles (fetching the queries, filling the pipeline, writing the result) in the same
// unit; an item's units are the extra ones first and then its tiles. Within a sequence, items go
// key-value head by key-value head and then by token tile, so that workers that run side by side
// read the same keys.
//
// All the items' units laid end to end are units 0 .. W-1, and worker w (a CTA) takes the units
// [w * per, (w + 1) * per) with per = ceil(W / workers). Prompts of any lengths, causal triangles
// and long caches with few rows are so balanced by one rule that needs no lengths on the host:
// every worker evaluates it for itself from the lengths in device memory. An item that a boundary
// cuts is computed in pieces, each with its own running maximum and sum, that are joined afterwards
// (attn_combine.cu), always in the same order. Where an item is small beside a worker's share, the
// boundary moves to the item's nearer end instead: up to a quarter of a share at either end of a
// worker's range costs less than the pieces' way through memory.
//
// A worker holds at most two pieces: one of an item that an earlier worker began (its first
// segment), and one of an item that it begins and a later worker finishes (its last segment).
#pragma once

#include <cstdint>

namespace engram {

constexpr int32_t kTileKeys = 128;   // keys per unit
// Items up to this size may be left whole. With 0, never: 14 prompts of 0-801 tokens 47.3 us instead
// of 44.5, chunks of five drafted tokens over 16 caches 40.4 instead of 39.2, long prompts the same.
constexpr int32_t kWholeUnits = 8;

struct AttnPlan {
  const int32_t* cu;       // [n_seqs + 1] first token of each sequence, and the end
  const int32_t* kv_len;   // [n_seqs] positions in the cache; null: keys are the tokens themselves
  int32_t n_seqs;
  int32_t total;           // tokens in q
  int32_t kv_cap;          // positions that a sequence's page table can hold
  int32_t kv_heads;
  int32_t tokens;          // query tokens per item
  int32_t workers;
  int32_t extra;           // units of an item beside its tiles
};

// One sequence: tokens [q0, q0 + n), of which token t sees the keys [0, max(0, m - n + t + 1)).
struct AttnSeq {
  int32_t q0, n, m;
};

__host__ __device__ inline int32_t attn_clamp(int32_t v, int32_t lo, int32_t hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

// Lengths come from device memory and are clamped to what the tensors hold.
__host__ __device__ inline AttnSeq attn_seq(const AttnPlan& p, int32_t b) {
  AttnSeq s;
  s.q0 = attn_clamp(p.cu[b], 0, p.total);
  s.n = attn_clamp(p.cu[b + 1], s.q0, p.total) - s.q0;
  s.m = p.kv_len ? attn_clamp(p.kv_len[b], 0, p.kv_cap) : s.n;
  return s;
}

__host__ __device__ inline int32_t attn_items(const AttnPlan& p, const AttnSeq& s) {
  return (s.n + p.tokens - 1) / p.tokens;
}

// Keys that the last token of token tile rt sees, and the tiles they fill (at least one).
__host__ __device__ inline int32_t attn_keys(const AttnPlan& p, const AttnSeq& s, int32_t rt) {
  const int64_t last = int64_t(rt + 1) * p.tokens;
  const int32_t x = s.m - s.n + (last < s.n ? static_cast<int32_t>(last) : s.n);
  return x > 0 ? x : 0;
}
__host__ __device__ inline int32_t attn_cost(const AttnPlan& p, const AttnSeq& s, int32_t rt) {
  const int32_t t = (attn_keys(p, s, rt) + kTileKeys - 1) / kTileKeys;
  return t > 0 ? t : 1;
}

// sum_{i < n} floor((a i + b) / kTileKeys), by the Euclidean reduction of the lattice-point count:
// take out what both a and b hold of the divisor, then exchange the roles of a and the divisor.
// a n + b stays below 2^32 (a < 2^8 after the first step, n < 2^24). One turn of the loop where a
// divides kTileKeys, none where it is a multiple.
__host__ __device__ inline uint64_t attn_floor_sum(uint32_t n, uint32_t a, uint32_t b) {
  uint32_t m = kTileKeys;
  uint64_t sum = (static_cast<uint64_t>(n) * (n - 1) / 2) * (a / kTileKeys) +
                 static_cast<uint64_t>(n) * (b / kTileKeys);
  a %= kTileKeys;
  b %= kTileKeys;
#pragma unroll 1
  for (uint32_t y = a * n + b; y >= m && n > 0; y = a * n + b) {
    n = y / m;
    b = y % m;
    const uint32_t t = a;
    a = m;
    m = t;
    sum += (static_cast<uint64_t>(n) * (n - 1) / 2) * (a / m) + static_cast<uint64_t>(n) * (b / m);
    a %= m;
    b %= m;
  }
  return sum;
}

// a / b for a >= 0, b > 0: in 32 bits where they are enough, else bit by bit (few instructions count
// for more than a case that hardly comes up).
__host__ __device__ inline int64_t attn_div(int64_t a, int64_t b) {
  if (((a | b) >> 31) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  uint64_t q = 0, r = 0;
#pragma unroll 1
  for (int i = 62; i >= 0; --i) {
    r = r << 1 | (static_cast<uint64_t>(a) >> i & 1u);
    q <<= 1;
    if (r >= static_cast<uint64_t>(b)) {
      r -= b;
      q |= 1u;
    }
  }
  return static_cast<int64_t>(q);
}

// Units of the token tiles 0 .. k-1 of one key-value head (k <= attn_items).
__host__ __device__ inline int64_t attn_units_before(const AttnPlan& p, const AttnSeq& s,
                                                     int32_t k) {
  if (k <= 0) return 0;
  int64_t u = static_cast<int64_t>(k) * p.extra;
  if (static_cast<int64_t>(k) * p.tokens >= s.n)   // the last one may hold fewer tokens
    u += attn_cost(p, s, --k);
  if (k == 0) return u;
  const int32_t a = s.m - s.n;
  int32_t z = a < 0 ? -a / p.tokens : 0;   // tiles that see nothing: one unit each
  if (z > k) z = k;
  u += z;
  if (k == z) return u;
  return u + static_cast<int64_t>(attn_floor_sum(
                 static_cast<uint32_t>(k - z), p.tokens,
                 static_cast<uint32_t>(a + (z + 1) * p.tokens + kTileKeys - 1)));
}

// Units of one of the sequence's key-value heads.
__host__ __device__ inline int64_t attn_head_units(const AttnPlan& p, const AttnSeq& s) {
  return attn_units_before(p, s, attn_items(p, s));
}

__host__ __device__ inline int64_t attn_share(const AttnPlan& p, int64_t units) {
  return attn_div(units + p.workers - 1, p.workers);
}

// Whether an item of `units` units is left whole where the share is `per`.
__host__ __device__ inline bool attn_whole(int32_t units, int64_t per) {
  return units <= kWholeUnits && 2 * units <= per;
}

// A stretch of one item's key tiles, [tile0, tile1) of `cost`.
struct AttnSegment {
  int32_t b, h;
  int32_t tile0, tile1, cost;
  int32_t q0;          // first token of its sequence
  int32_t token0;      // first token of the item in q
  int32_t ntok;        // its tokens
  int32_t keys;        // that the item's last token sees
  int32_t first;       // that its first token sees: token i sees first + i; none if that is <= 0
  int32_t owner;       // the worker that begins it
  int32_t pieces;      // workers that hold a piece of it: owner, owner + 1, ... (at least 1)
  __host__ __device__ bool begins() const { return tile0 == 0; }
  __host__ __device__ bool ends() const { return tile1 == cost; }
};

// Walks a worker's segments in order. (b, h, rt, unit) is where its range begins and `left` the
// units in it.
struct AttnCursor {
  AttnSeq seq;
  int32_t items;  // token tiles of the sequence
  int32_t b, h, rt, unit;
  int32_t worker;
  int32_t per;    // the share, cut at 2^30 (an item is far smaller)
  int64_t left;

  __host__ __device__ bool next(const AttnPlan& p, AttnSegment& out) {
    if (left <= 0 || b >= p.n_seqs) return false;
    out.b = b;
    out.h = h;
    out.cost = attn_cost(p, seq, rt);
    const int32_t units = out.cost + p.extra;
    int32_t end = left >= units - unit ? units : unit + static_cast<int32_t>(left);
    if (end < units && attn_whole(units, per)) {   // the boundary moves to the nearer end
      if (2 * end <= units) {
        left = 0;
        return false;
      }
      left = units - unit;
      end = units;
    }
    out.tile0 = unit > p.extra ? unit - p.extra : 0;
    out.tile1 = end > p.extra ? end - p.extra : 0;
    out.keys = attn_keys(p, seq, rt);
    const int32_t t0 = rt * p.tokens;
    out.q0 = seq.q0;
    out.token0 = seq.q0 + t0;
    out.ntok = seq.n - t0 < p.tokens ? seq.n - t0 : p.tokens;
    out.first = seq.m - seq.n + t0 + 1;
    out.owner = worker;
    out.pieces = 1;
    if (unit > p.extra) {
      const int32_t before = (unit - p.extra + per - 1) / per;
      out.owner -= before;
      out.pieces += before;
    }
    if (end < units) out.pieces += (units - end + per - 1) / per;
    left -= end - unit;
    if (end == units) step(p);
    return out.tile1 > out.tile0;   // a range may end before the item's first tile
  }

  // To the next item.
  __host__ __device__ void step(const AttnPlan& p) {
    unit = 0;
    if (++rt < items) return;
    rt = 0;
    if (++h < p.kv_heads) return;
    h = 0;
#pragma unroll 1
    do {
      if (++b >= p.n_seqs) return;
      seq = attn_seq(p, b);
    } while (seq.n == 0);
    items = attn_items(p, seq);
  }

  // The range of worker `w` begins inside sequence b, in token tile `rt` of key-value head h, which
  // begins `in` units before it, and holds `units`.
  __host__ __device__ void start(const AttnPlan& p, int32_t w, int64_t share, int32_t b_, int32_t h_,
                                 int32_t rt_, int32_t in, int64_t units) {
    worker = w;
    per = share < (1 << 30) ? static_cast<int32_t>(share) : 1 << 30;
    b = b_;
    h = h_;
    rt = rt_;
    unit = in;
    left = units;
    seq = attn_seq(p, b);
    items = attn_items(p, seq);
    const int32_t all = attn_cost(p, seq, rt) + p.extra;
    if (unit > 0 && attn_whole(all, per)) {   // as the worker before has it
      if (2 * unit <= all) {
        left += unit;
        unit = 0;
      } else {
        left -= all - unit;
        step(p);
      }
    }
  }
};

}  // namespace engram
