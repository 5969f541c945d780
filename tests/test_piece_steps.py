"""Host-side replay of the waits of the paged forward's two MMA issuers (csrc/piece_steps.h): the header that
the kernel compiles, run on the CPU over many pieces.  A K/V barrier tells only the parity of its phase, so every
wait for ring index i has to be preceded by the knowledge that index i - NS has landed: from a wait of the same
issuer, or handed over with a turn.  And every slot is freed by two arrivals, after the waits of all who read it."""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "scaled_dot_product_fa2_b200", "csrc")

CHECK = r"""
#include <cstdio>
#include <cstdint>
#include <cstdlib>
#include <set>
#include <vector>
#include "piece_steps.h"

struct Event { char what; int i, n; };  // P: p, T: takes turn i, W: waits for tile i, M: multiply, F: frees i (n arrivals), H: hands over

template <int NS>
struct Record {
  std::vector<Event>& e;
  int in_slot[NS];  // ring index that the issuer last waited for there
  bool wrong;
  explicit Record(std::vector<Event>& events) : e(events), wrong(false) {
    for (int& i : in_slot) i = -1;
  }
  int tile(int slot) { return slot < 0 ? -1 : in_slot[slot]; }
  bool p_ready() { e.push_back({'P', 0, 0}); return true; }
  bool turn_ready(int s) { e.push_back({'T', s, 0}); return true; }
  bool tile_ready(int i, int slot) {
    wrong |= slot != i % NS;
    in_slot[slot] = i;
    e.push_back({'W', i, 0});
    return true;
  }
  void multiply(int, int vs, int ks) { e.push_back({'M', tile(vs), tile(ks)}); }
  void free_tile(int slot, int n) { e.push_back({'F', tile(slot), n}); }
  void hand_over() { e.push_back({'H', 0, 0}); }
};

static uint64_t state = 0x9E3779B97F4A7C15ull;
static int below(int n) {
  state ^= state >> 12; state ^= state << 25; state ^= state >> 27;
  return static_cast<int>(((state * 0x2545F4914F6CDD1Dull) >> 33) % n);
}

// 0: sound; else what is wrong
template <int NS>
static int replay(int pieces, int kind) {
  std::vector<Event> e[2];
  int it_base = 0, seg[2] = {0, 0};
  for (int r = 0; r < pieces; ++r) {
    sdpa::PieceSteps s;
    const bool thin = kind == 2 ? below(2) : kind == 1;
    const int steps = below(4) == 0 ? below(3) : below(40);
    s.thin = thin;
    s.it_base = it_base;
    s.n0 = thin ? (steps + 1) / 2 : (steps > 0 ? steps - below(2 < steps ? 2 : steps) : 0);
    s.n1 = thin ? steps / 2 : steps;
    it_base += 2 * steps;
    for (int t = 0; t < 2; ++t) {
      Record<NS> op(e[t]);
      if (!sdpa::walk_piece<NS>(op, s, t, seg[t]) || op.wrong) return 1;
    }
  }
  if (seg[0] != seg[1]) return 2;
  std::set<int> known[2], handed[2];  // tiles known to have landed; what the last hand-over carried
  std::vector<std::vector<std::set<int>>> passes(2);
  std::vector<int> frees(it_base, 0);
  std::vector<char> landed(it_base, 0);
  size_t at[2] = {0, 0};
  int issued = 0;
  std::vector<std::set<int>> mine(2);
  while (at[0] < e[0].size() || at[1] < e[1].size()) {
    bool moved = false;
    while (issued < it_base && (issued < NS || frees[issued - NS] == 2)) { landed[issued++] = 1; moved = true; }
    for (int t = 0; t < 2; ++t) {
      while (at[t] < e[t].size()) {
        const Event& x = e[t][at[t]];
        if (x.what == 'T') {
          if (static_cast<int>(passes[1 - t].size()) <= x.i) break;
          for (int i : passes[1 - t][x.i]) known[t].insert(i);
        } else if (x.what == 'W') {
          if (x.i >= NS && !known[t].count(x.i - NS)) return 10;  // may be answered by the phase before
          if (frees[x.i] == 2) return 11;                         // may be past already
          if (!landed[x.i]) break;
          known[t].insert(x.i);
          mine[t].insert(x.i);
        } else if (x.what == 'M') {
          for (int i : {x.i, x.n})
            if (i >= 0 && !mine[t].count(i)) return 12;  // reads what it did not wait for
        } else if (x.what == 'F') {
          if (!mine[t].count(x.i)) return 13;
          frees[x.i] += x.n;
        } else if (x.what == 'H') {
          // (old tiles do not matter any more)
          std::set<int> recent(known[t].lower_bound(issued - 4 * NS), known[t].end());
          passes[t].push_back(recent);
        }
        ++at[t];
        moved = true;
      }
    }
    if (!moved) return 20;  // nobody can go on
  }
  for (int i = 0; i < it_base; ++i)
    if (frees[i] != 2) return 21;
  return 0;
}

template <int NS>
static int check() {
  for (int kind = 0; kind < 3; ++kind)
    for (int i = 0; i < 100; ++i) {
      const int r = replay<NS>(1 + below(30), kind);
      if (r != 0) {
        std::printf("NS=%d kind=%d: %d\n", NS, kind, r);
        return 1;
      }
    }
  return 0;
}

int main() { return (CHECKS) != 0; }
"""


def stages():
    """Slots of the K/V ring for head_dim 128 and 64, from the launch code."""
    with open(os.path.join(CSRC, "sdpa_b200.cu")) as f:
        text = f.read()
    return [int(re.search(rf"\b{name} = (\d+)", text).group(1)) for name in ("kStagesD128", "kStagesD64")]


def test_no_wait_of_an_issuer_can_be_answered_by_the_phase_before(tmp_path):
    src = tmp_path / "piece_steps_check.cpp"
    # the rings that the kernels have, and other lengths
    rings = stages() + [4, 6, 7, 9, 10, 12]
    src.write_text(CHECK.replace("CHECKS", " + ".join(f"check<{n}>()" for n in rings)))
    exe = tmp_path / "piece_steps_check"
    try:
        subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True,
                       capture_output=True, text=True)
    except FileNotFoundError:
        pytest.skip("no host C++ compiler")
    proc = subprocess.run([str(exe)], capture_output=True, text=True)
    assert proc.returncode == 0, proc.stdout
