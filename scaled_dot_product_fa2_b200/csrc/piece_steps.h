// piece_steps.h -- the order in which an MMA issuer of the paged forward waits,
// multiplies and frees ring slots over the segments of one piece of a unit.
//
// Two issuers (t = 0, 1) walk the same n_max + 1 segments and take turns: tile 0
// segment k, tile 1 segment k, tile 0 segment k + 1, ...  Segment k of tile t is
// O_t += P_t(k-1) V (its key tile k - 1) and S_t(k) = Q_t K^T (its key tile k).
// In a pair both read every key tile; in a thin piece tile t's k-th key tile is
// 2 k + t and only its issuer waits for it, and frees it for both.
//
// A K/V barrier tells only the parity of its phase: a wait for ring index i is
// answered at once, and wrongly, where the copy of i - NS, which had the slot before,
// has not landed yet.  So an issuer may wait for i only when it knows that
// i - NS has landed: it waited for it itself, or the other issuer did before it
// handed over a turn that this one took.  What it waited for itself in this piece
// it may ask for before its turn; with an odd number of slots the slots of a thin
// piece alternate between the issuers, and then (and at a piece's start) the wait
// stands behind the turn.  All waits behind the turn cost: 2200 -> 2270 us for a
// 16384-token prompt (32 / 8 heads, d = 128), 105.6 -> 108.6 for 129 tokens behind 32639.
// Host and device code share this header.
#pragma once
#include "fastdiv.h"

namespace sdpa {

struct PieceSteps {
  int n0, n1;    // key tiles of tile 0 and tile 1
  bool thin;     // the tiles take key tiles in turn
  int it_base;   // ring index of the piece's first K tile (K and V of a key tile follow one another)
};

// Segments of one piece for issuer t; `seg` counts them over all pieces.  Operations:
//   p_ready()                  wait for P_t of the key tile before
//   turn_ready(seg)            wait until the other issuer handed over
//   tile_ready(i, slot)        wait for ring index i, which is in `slot`
//   multiply(k, vs, ks)        issue segment k's products with V in slot vs and K in slot ks (-1: none)
//   free_tile(slot, times)     when the products so far are done, the slot is free (`times` arrivals)
//   hand_over()                the other issuer's turn
// The waits return false where they gave up, and so does this.
template <int NS, class Ops>
SDPA_HOST_DEVICE bool walk_piece(Ops& op, const PieceSteps& s, int t, int& seg) {
  const int nt = t ? s.n1 : s.n0;
  const int n_max = s.n0 > s.n1 ? s.n0 : s.n1;
  const int n_slots = s.thin ? nt : n_max;  // key tiles whose slots this issuer frees
  const int times = s.thin ? 2 : 1;
#pragma unroll 1
  for (int k = 0; k <= n_max; ++k, ++seg) {
    const int v = k >= 1 && k <= n_slots ? s.it_base + 2 * (s.thin ? 2 * (k - 1) + t : k - 1) + 1 : -1;
    const int kt = k < n_slots ? s.it_base + 2 * (s.thin ? 2 * k + t : k) : -1;
    // whether the slot's tile before (of ring index b + it_base) is one that this issuer waited for in this piece
    const int vb = v - NS - s.it_base, kb = kt - NS - s.it_base;
    const bool v_early = vb >= 0 && (!s.thin || ((vb >> 1) & 1) == t);
    const bool k_early = kb >= 0 && (!s.thin || ((kb >> 1) & 1) == t);
    // slots: once, not in each operation (a prompt of 16384 tokens 2186 -> 2136 us)
    const int vs = v >= 0 ? v % NS : -1, ks = kt >= 0 ? kt % NS : -1;
    if (v_early && !op.tile_ready(v, vs)) return false;
    if (k_early && !op.tile_ready(kt, ks)) return false;
    if (k >= 1 && k - 1 < nt && !op.p_ready()) return false;
    if ((t == 1 || seg >= 1) && !op.turn_ready(t == 1 ? seg : seg - 1)) return false;
    if (v >= 0 && !v_early && !op.tile_ready(v, vs)) return false;
    if (kt >= 0 && !k_early && !op.tile_ready(kt, ks)) return false;
    op.multiply(k, vs, ks);
    if (v >= 0) op.free_tile(vs, times);
    if (kt >= 0) op.free_tile(ks, times);
    op.hand_over();
  }
  return true;
}

}  // namespace sdpa
