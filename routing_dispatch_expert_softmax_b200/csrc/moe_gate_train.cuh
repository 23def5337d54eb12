// Workspace layouts of the calls that train the gate, and the plan of the router's
// backward (host code).  Apart from moe_common.cuh: the expert GEMMs' recorded traffic
// belongs to that file as it is.
#pragma once

#include <algorithm>

#include "moe_common.cuh"

namespace moe {

// The workspace header's words after those of moe_common.cuh: tickets of the balance
// loss and of the gradient norm, each back to 0 at the end of every call.
enum : int { kBalanceTicket = 3, kGradTicket = 4 };

// Workspace of the gate's training calls (moe_workspace_size_bwd).  The balance
// loss and the router's backward each use the region after the header as their
// own scratch; nothing in it outlives a call.
constexpr int kMaxSeqs = 65535;
struct BwdLayout {
  // balance loss: blocks of `chunk` tokens, one partial per (block, sequence)
  // pair that meets (at most blocks + S of them)
  int chunk;
  size_t prob, count, z, n, term, zterm;
  // router backward: bf16 planes of dlogits (router_planes), dlogits [T][2][cp] and w_g
  // [d][2][cp] in two fp16 parts (cp = E rounded up to 64) with the roots of the factors
  // that undo their rows' scaling, column sums of every plane_rows tokens, and (last)
  // partial weight gradients of the token ranges
  int cp, plane_rows;
  size_t dl_planes, dl_half, w_half, dl_back, w_back, db_part, dw_part;
  size_t balance, rest;  // the bytes for the balance loss, and of all but dw_part
};

// How the router's backward lays dL's three bf16 planes out for dW's 128-row MMA
// operand: above 64 experts a plane of its own each (three MMAs for each K step);
// up to 64, side by side in rows of (hi | mid | lo | 0) x 64 (two MMAs); up to
// 32, of x 32 (one).  Side by side, a plane's rows of the product are apart, so a
// tile is `parts` partial weight gradients, and a kernel has to add them: up to 256
// tokens that costs more (2.5 us) than the MMAs.
struct RouterPlanes {
  int sets, parts, width;  // MMAs for each K step; partials; columns of one plane
};
inline RouterPlanes router_planes(int E, int T) {
  if (E <= 32 && T > 256) return {1, 3, 32};
  if (E <= 64 && T > 256) return {2, 2, 64};
  return {3, 1, (int)((E + 63) / 64 * 64)};
}

// Times in us that the router's backward plans with, as measured: a 64-token block
// of a 128 x 256 tile of dW (the MMAs, or for one set the 32 KB of x); a 128 x 256
// tile of dx (its 64 KB of output up to 64 experts, the MMAs from there on, and above
// 128 W's tiles too, which the shared memory then does not keep; alone a tile takes a
// quarter more, but with this factor the calls of both products took least, over
// eleven shapes); an item's start and end.
inline double router_dw_block_us(int sets) {
  return sets == 3 ? 1.1 : sets == 2 ? 0.85 : 0.68;
}
inline double router_dx_tile_us(int E) {
  const int kx = (E + 63) / 64;
  return kx == 1 ? 1.6 : kx == 2 ? 2.1 : 1.15 * kx;
}
constexpr double kRouterItemUs = 2.0;

// Adding up a partial costs its share of L2's bandwidth and a step of a chain of loads
// (eight of them at a time from 16 partials on).
inline double router_partial_us(const moe_shape& s, int parts, long long ranges) {
  const long long n = parts * ranges;
  return 8.0 * n * s.d * s.E / 1e7 + (n > 1 ? 2.5 : 0.0) + 0.1 * (n < 16 ? n : n / 8.0);
}

// The tokens of dW are cut into ranges: more of them fill the SMs, but each
// writes partials that are read again.  The time of `r` ranges: all work over
// 148 SMs, but no less than the longest SM's dW items; a share of that longest,
// since long items leave the rest uneven; and the partials'.  The r with the least
// time is taken; what is returned is the 64-token blocks of one range.  Of twelve shapes
// from 300 to 16384 tokens and 32 to 1024 experts the plan was within 4% of the best
// range count in all but 1024 x 2048 x 128 without dx (8 ranges 13.1 us, 16 planned 14.2)
// and 2048 x 2048 x 128 with it (16 ranges 19.5, 11 planned 21.7).
inline int router_range_blocks(const moe_shape& s, bool dx) {
  const RouterPlanes pl = router_planes(s.E, s.T);
  const double kb = router_dw_block_us(pl.sets);
  const long long cols = (s.d + 255) / 256;
  const long long tiles = cols * (pl.sets == 3 ? (s.E + 127) / 128 : 1);
  const long long blocks = ((long long)s.T + 63) / 64;
  const double dx_us = dx ? (double)((s.T + 127) / 128) * cols * router_dx_tile_us(s.E) : 0.0;
  long long best = std::max(1LL, blocks);
  double least = 0.0;
  // (1 to 8 one by one, then steps of an eighth: this runs on the host in every call)
  for (long long r = 1; r <= std::min(blocks, 148LL); r += std::max(1LL, r / 8)) {
    const long long per = (blocks + r - 1) / r, n = (blocks + per - 1) / per;
    const double waves = (double)((tiles * n + 147) / 148);
    const double longest = waves * (per * kb + kRouterItemUs);
    const double all = (tiles * (blocks * kb + n * kRouterItemUs) + dx_us) / 148;
    const double us =
        std::max(longest, all) + 0.15 * longest + router_partial_us(s, pl.parts, n);
    if (r == 1 || us < least) best = per, least = us;
  }
  return (int)best;
}

inline BwdLayout bwd_layout(const moe_shape& s, int S) {
  BwdLayout L{};
  const long long T = s.T, d = s.d, E = s.E;
  size_t o = 256;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  // One sequence of up to 64 tokens: one block.  Else 32 tokens a block (4 for each
  // warp), or the tokens of an average sequence (a block takes the sequences in its
  // tokens one after the other), until the SMs are full, with four blocks (three above
  // 256 experts, two above 512) each.
  const long long nblk = E <= 256 ? 592 : E <= 512 ? 444 : 296;
  const long long least = std::min(32LL, std::max(1LL, T / S));
  L.chunk = S == 1 && T <= 64 ? 64 : (int)std::max(least, (T + nblk - 1) / nblk);
  const size_t slots = (size_t)((T + L.chunk - 1) / L.chunk) + S;
  L.prob = take(sizeof(float) * slots * E);
  L.count = take(sizeof(int) * slots * E);
  L.z = take(sizeof(float) * slots);
  L.n = take(sizeof(int) * slots);
  L.term = take(sizeof(double) * (size_t)S * ((E + 31) / 32));
  L.zterm = take(sizeof(double) * S);
  L.balance = o;
  o = 256;
  L.cp = (int)align_up(E, 64);
  // up to 64 tokens one block, whose column sums need no second kernel
  L.plane_rows = T <= 64 ? 64 : (int)std::max(32LL, (T + 591) / 592);
  const RouterPlanes pl = router_planes(s.E, s.T);
  L.dl_planes = take(2 * (size_t)T * pl.width * (pl.sets == 3 ? 3 : 4));
  L.dl_half = take(4 * (size_t)T * L.cp);
  L.w_half = take(4 * (size_t)d * L.cp);
  L.dl_back = take(2 * (size_t)T);
  L.w_back = take(2 * (size_t)d);
  L.db_part = take(sizeof(float) * (size_t)((T + L.plane_rows - 1) / L.plane_rows) * E);
  L.dw_part = o;
  L.rest = std::max(L.balance, o);
  return L;
}

// The layout's bytes.  Apart from it: the search for the ranges takes the host a
// microsecond or two, and only their own call needs them.
inline size_t bwd_bytes(const moe_shape& s, int S) {
  const BwdLayout L = bwd_layout(s, S);
  const long long per = std::min(router_range_blocks(s, false), router_range_blocks(s, true));
  const long long ranges = ((s.T + 63LL) / 64 + per - 1) / per;
  const int parts = router_planes(s.E, s.T).parts;
  const size_t part = ranges * parts > 1 ? sizeof(float) * (size_t)ranges * parts * s.d * s.E : 0;
  return std::max(L.rest, align_up(L.dw_part + part, 256));
}

}  // namespace moe
