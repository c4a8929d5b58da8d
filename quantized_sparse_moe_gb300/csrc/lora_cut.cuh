// How a call of lora.cu is cut up over the device.  Plain host code: what the
// device holds comes in as numbers.
#pragma once

#include <cstdint>

namespace qsm {
namespace lora {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 64;               // tokens, at most
constexpr int kMostCounted = 1023;      // adapters whose tokens a CTA counts
constexpr int kMostGrouped = 1 << 14;   // tokens that a CTA looks through; their ids fit where the partial sums will lie

// Whether the tokens of an adapter make items, wherever they are.
inline bool grouped(long long T, int n) { return T > kTile && T <= kMostGrouped && n <= kMostCounted; }

struct Cut {
  int cs, lanes, parts;  // CTAs of a cluster, slots' lanes (or clusters for items), column parts
  int room;              // items that run at once
  long long ctas;        // 0: nothing fits
};

// A launch in one wave if it can be.  Clusters of 8 CTAs, fewer when there are more
// slots or items than such clusters fit on the device at once (a GB300, two CTAs an SM: 36
// of 8, 74 of 4, 152 of 2, 304 of 1).  Slots have a cluster each while they fit; and columns come
// in parts while SMs would be idle.
// Items are of 16 tokens with clusters of 8, up to 32 with 4 or 2, else what fits: less of a
// product's latency hangs on one item (us, clusters of 8, 4, 2, 1; six to sixteen adapters: 300 tokens
// 2048 x 2048 10.0 10.1 11.0 12.4; 904 1216 x 734 16 10.1 11.0 10.5; 1714 496 x 248 19 11.0 10.0 8.3; 4096
// 2048 x 8192 57 42.0 41.6 51: of the third, whose products are short, single CTAs would have the least;
// the rule does not go by K and N).  In launches that follow one another closely not all those clusters
// find room beside the early ones of the next launch (1024 x 1024, rank 16, us: 30 of 8 9.2, 31
// 11.5, 36 15.2; 70 of 4 10.4, 74 13.8): the shares left out below.
// Items against tiles of 64 tokens as they follow one another, whose adapters a cluster takes in
// turn (us; 2048 x 8192, rank 32): 4096 tokens of six adapters in six runs 41 against 54, in no
// order 42 against 92, of 64 adapters 53 against 444; 16384 in six runs 128 against 176.
// Beyond kMostGrouped tokens, or kMostCounted adapters, every CTA would look through too much, and it
// is tiles: 2048 x 2048, 32768 in six runs 131 against 188, but in no order 224 against 193.
// The cut knows the adapters that are loaded, not those that the ids name (they are on the device): 300 tokens
// of one adapter, 2048 x 8192, rank 32, take 11.6 us where it is the only one, 18.5 among 64, 36.8 among 256;
// 64 tokens 13.5, 25.7, 25.8; 4096 40.7, 49.9, 50.5, among 1000 77.3.
//
// singles: single CTAs that the device holds; clusters(cs): clusters of cs.
template <typename Clusters>
Cut cut(bool items, long long T, int n, int N, long long singles, Clusters clusters) {
  Cut c = {};
  const int tile = T < kTile ? (int)T : kTile;
  const auto resident = [&](int cs) -> long long {
    if (cs == 1) return singles;
    const long long r = clusters(cs);
    return !items ? r : cs == 8 ? r - r / 6 : cs == 4 ? r - r / 18 : r;
  };
  const auto tiles_of = [&](int t) { return (T + t - 1) / t; };
  const auto items_of = [&](int t) { return tiles_of(t) + (n + 1ll < T ? n + 1 : T); };  // at most
  const int one = n + 1ll < tile ? n + 1 : tile;  // slots of a tile at most
  c.cs = 8;
  while (c.cs > 1 && (items ? items_of(c.cs == 8 ? 16 : 32) : T <= kTile ? one : tiles_of(kTile)) > resident(c.cs)) c.cs /= 2;
  const long long room = resident(c.cs);
  if (room < 1) return c;
  const long long tiles = items ? 1 : tiles_of(tile);
  long long lanes = tiles * one <= room ? one : room / tiles < 1 ? 1 : room / tiles;
  if (items) lanes = items_of(16) < room ? items_of(16) : items_of(kTile) > room ? items_of(kTile) : room;
  c.lanes = (int)lanes;
  c.parts = 1;
  const int chunks = (N + 31) / 32;
  while (tiles * lanes * c.parts * 2 <= room && c.parts * 2 * c.cs * kWarps <= chunks) c.parts *= 2;
  c.room = (int)(lanes < room / c.parts ? lanes : room / c.parts);
  c.ctas = tiles * lanes * c.parts * c.cs;
  return c;
}

}  // namespace lora
}  // namespace qsm
