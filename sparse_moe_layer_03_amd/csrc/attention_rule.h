// How an attention call is cut into workgroups: a rule on its sizes alone, in plain C++.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "moe.h"

namespace moe {
namespace attn {

struct Plan {
  int rows;     // of a workgroup: 32, whose keys are dealt over its waves, 128 or 256
  bool stream;  // equal shares of all keys instead of one workgroup per row tile
  int grid, min_units;
};
inline Plan plan_of(int type, int T, int S, int Hq, int Hkv, int D, int64_t max_keys, int window) {
  const int64_t G = Hq / Hkv;
  // a sequence's rows, T at most, see no more than this of its keys
  if (window > 0) max_keys = std::min(max_keys, (int64_t)window + T + 63);
  Plan p;
  // An average over the sequences, empty ones too: their lengths are on the device, and a captured call serves any.
  // Where they differ much it is no good guide, us: one prompt of 1024 among 256 slots, 32 heads over 4, 56 (31 by
  // itself); a single token behind 131072 keys beside 62 short ones and 2048 prompt tokens, in a tile of 128 rows that is
  // not shared out, 2503 (55 by itself; the others 78 together, 64 and 44 apart).
  const bool few = T * G <= 32 * (int64_t)S;
  auto items_of = [&](int rows) { return (T * G + rows - 1) / rows * Hkv; };
  // a launch holds fewer than 2^32 threads, 512 each in workgroups of 256 rows (256 in the others: always)
  const bool wide = D == 128 && type == MOE_BF16 && items_of(256) >= 512 && (T * G / 256 + S) * Hkv < 1 << 23;
  p.rows = few ? 32 : wide ? 256 : 128;
  const int unit = few ? (D == 64 ? 256 : 128) : 64;
  const int64_t tiles = T * G / p.rows + S;  // or fewer
  const int64_t units = (max_keys + 63 + unit - 1) / unit;
  // Row tiles of 128 to share out below 256 of them, for long contexts only: what is shared has to be joined, and the
  // shares count masked keys.  Shared / not, us: prompts of 512 and 1024 (128 and 256 tiles) 30 / 19 and 53 / 31; 4
  // chunks of 128 behind 1024 (128 tiles) 46 / 33, 2 of 256 behind 4096 75 / 103, one of 512 behind 8192 at D 64
  // 76 / 165.  Up to 64 tiles leave three quarters of the CUs idle: shorter contexts too, in shares of half the size
  // (shares of 4 units / of 8 / not: a prompt of 1024, 32 tiles, 20 / 24 / 29, at D 256 33 / 45 / 56; 2 chunks of 128
  // behind 1700, 16 tiles, 25 / 31 / 48; from 6 units on instead of 12, 32 tiles of 9 units, 24 / - / 20).
  const bool idle = items_of(128) <= 64;
  p.min_units = few ? 1 : idle ? 4 : 8;
  // Keys that a tile's rows, of at most as many tokens, see.  (With the whole context in its place, us: 2 chunks of 431
  // behind 84897, window 129, D 256 60 and now 26; 6 drafts of 8, window 1, 52 and 10; 64 decode requests, window 128,
  // 17 and 11.)
  const int64_t seen = window > 0 ? std::min(max_keys, (int64_t)window + p.rows) : max_keys;
  p.stream = few ? seen > 2 * unit : items_of(128) < 256 && seen + 63 > 64 * (idle ? 12 : 32);
  const int64_t all = tiles * Hkv * (p.stream ? (units + p.min_units - 1) / p.min_units : 1);
  const int64_t most = D == 256 ? 256 : 512;
  p.grid = (int)(p.stream && all > most ? most : all);
  return p;
}

}  // namespace attn
}  // namespace moe
