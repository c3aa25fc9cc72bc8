"""Host check of how the attention kernels share out their work (no GPU): the header is compiled
with g++ into a program that walks every worker's segments for many batches and checks that they
tile every item's key tiles exactly once and in order, that small items are whole, that a worker
holds at most one piece it continues and one it begins, that all pieces of a cut item name the same
first worker and the same number of pieces, and that the closed forms equal plain sums."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "deepseek_v4_engram_gb300", "csrc")

PROGRAM = r"""
#define __host__
#define __device__
#include "attn_plan.cuh"
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>
using namespace engram;

static long check(AttnPlan p) {
  long bad = 0;
  // plain sums against the closed forms
  int64_t total = 0;
  std::vector<int64_t> first(p.n_seqs);
  for (int b = 0; b < p.n_seqs; ++b) {
    AttnSeq s = attn_seq(p, b);
    first[b] = total;
    int64_t u = 0;
    for (int rt = 0; rt < attn_items(p, s); ++rt) {
      if (attn_units_before(p, s, rt) != u) ++bad;
      long x = s.m - s.n + std::min<long>((long)(rt + 1) * p.tokens, s.n);
      long t = x <= 0 ? 1 : (x + kTileKeys - 1) / kTileKeys;
      if (attn_cost(p, s, rt) != t) ++bad;
      u += t + p.extra;
    }
    if (attn_head_units(p, s) != u) ++bad;
    total += u * p.kv_heads;
  }
  const int64_t per = attn_share(p, total);
  if (per * p.workers < total) ++bad;
  std::map<std::tuple<int, int, int>, int> done;     // item -> tiles done
  std::map<std::tuple<int, int, int>, std::pair<int, int>> cut;   // cut item -> owner, pieces so far
  std::map<std::tuple<int, int, int>, int> pieces;
  for (int w = 0; w < p.workers; ++w) {
    const int64_t u0 = per * w;
    if (u0 >= total) break;
    int b = p.n_seqs - 1;
    while (first[b] > u0 || attn_head_units(p, attn_seq(p, b)) == 0) --b;
    AttnCursor c;
    const AttnSeq at = attn_seq(p, b);
    const int64_t head = attn_units_before(p, at, attn_items(p, at)), pos = u0 - first[b];
    int rt = 0;
    while (rt + 1 < attn_items(p, at) && attn_units_before(p, at, rt + 1) <= pos % head) ++rt;
    c.start(p, w, per, b, pos / head, rt, pos % head - attn_units_before(p, at, rt),
            total - u0 < per ? total - u0 : per);
    AttnSegment s;
    bool was_last = false;
    int n = 0;
    int64_t units = 0;
    while (c.next(p, s)) {
      if (was_last) ++bad;                       // a piece that does not end is a worker's last
      AttnSeq q = attn_seq(p, s.b);
      auto key = std::make_tuple(s.b, s.h, (s.token0 - q.q0) / p.tokens);
      if (done[key] != s.tile0 || s.tile1 <= s.tile0 || s.tile1 > s.cost) ++bad;
      done[key] = s.tile1;
      if (!s.begins() && n != 0) ++bad;          // one that an earlier worker began is its first
      if (!(s.begins() && s.ends())) {
        // an item that counts as small is whole; the others agree on who holds their pieces
        if (attn_whole(s.cost + p.extra, per)) ++bad;
        if (s.begins()) cut[key] = {w, 0};
        if (s.owner != cut[key].first || s.owner + cut[key].second != w) ++bad;
        ++cut[key].second;
        if (s.begins()) pieces[key] = s.pieces;
        if (s.pieces != pieces[key]) ++bad;
        if (s.ends() != (cut[key].second == s.pieces)) ++bad;
      }
      was_last = !s.ends();
      const int t0 = s.token0 - q.q0;
      if (t0 % p.tokens || s.q0 != q.q0 || s.ntok < 1 || s.ntok > p.tokens || t0 + s.ntok > q.n ||
          (s.ntok < p.tokens && t0 + s.ntok != q.n)) ++bad;
      if (s.first != q.m - q.n + t0 + 1 || s.keys != std::max(0, s.first + s.ntok - 1)) ++bad;
      units += s.tile1 - s.tile0 + (s.begins() ? p.extra : 0);
      ++n;
    }
    // beyond its share, a worker has at most half a small item at each end
    if (units > per + std::min<int64_t>(kWholeUnits, per / 2) + p.extra) ++bad;
  }
  for (int b = 0; b < p.n_seqs; ++b) {
    AttnSeq s = attn_seq(p, b);
    for (int h = 0; h < p.kv_heads; ++h)
      for (int rt = 0; rt < attn_items(p, s); ++rt)
        if (done[std::make_tuple(b, h, rt)] != attn_cost(p, s, rt)) ++bad;
  }
  for (auto& o : cut) if (o.second.second != pieces[o.first]) ++bad;
  return bad;
}

int main() {
  srand(3);
  long bad = 0, cases = 0;
  const int lens[] = {0, 1, 2, 5, 16, 17, 64, 127, 128, 129, 300, 777, 2100};
  for (int rep = 0; rep < 3000; ++rep) {
    AttnPlan p{};
    p.n_seqs = 1 + rand() % 6;
    std::vector<int> cu(p.n_seqs + 1, 0), kv(p.n_seqs);
    for (int b = 0; b < p.n_seqs; ++b) {
      cu[b + 1] = cu[b] + lens[rand() % 13];
      kv[b] = lens[rand() % 13] * (rand() % 3 == 0 ? 40 : 1);
      if (rand() % 3) kv[b] += cu[b + 1] - cu[b];
    }
    p.total = cu.back();
    if (rand() % 7 == 0) cu[rand() % (p.n_seqs + 1)] = (rand() % 4000) - 1000;   // not ascending
    p.cu = cu.data();
    p.kv_len = rand() % 2 ? kv.data() : nullptr;
    p.kv_cap = 1 << (8 + rand() % 10);
    p.kv_heads = 1 + rand() % 4;
    const int toks[] = {1, 2, 3, 16, 36, 51, 64, 85, 128, 256};
    p.tokens = toks[rand() % 10];
    p.workers = 1 + rand() % 152;
    p.extra = rand() % 4;
    bad += check(p);
    ++cases;
  }
  // a very long cache: the sums pass 32 bits
  int cu[2] = {0, 1 << 20}, kv[1] = {1 << 29};
  AttnPlan p{cu, kv, 1, 1 << 20, 1 << 29, 128, 2, 152, 3};
  const int64_t u = attn_head_units(p, attn_seq(p, 0)) * p.kv_heads;
  long double want = 0;
  for (long r = 0; r < (1 << 19); ++r)
    want += ((1L << 29) - (1L << 20) + (r + 1) * 2 + 127) / 128 * 128.0L + 3 * 128.0L;
  if ((long double)u != want) ++bad;
  printf("cases=%ld bad=%ld\n", cases, bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_segments_tile_every_item_once(tmp_path):
    src = tmp_path / "check.cpp"
    src.write_text("#include <algorithm>\n" + PROGRAM)
    exe = tmp_path / "check"
    subprocess.run(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-I", CSRC, str(src),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and "runtime error" not in r.stderr, r.stdout + r.stderr
    assert dict(kv.split("=") for kv in r.stdout.split())["bad"] == "0"
