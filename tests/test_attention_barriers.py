"""The barriers between the threads of the decode attention (csrc/attn_tiles.h, attention_tc.cu), as
a model on the host: every order in which the issuing thread, the softmax threads and the products
can take their steps ends, and no wait lets its thread pass early."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mtp_block_draft_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <set>
#include <tuple>
#include <vector>
#include "attn_tiles.h"

enum Bar { S0, S1, P0, P1, Q, O, FIN, DRAINED, BARS };
enum Kind { WAIT, MAY_WAIT, ARRIVE, COMMIT };
struct Step {
  Kind kind;
  int bar;
  unsigned parity;
  int phase;  // a wait's: phases that have to be complete
};
typedef std::vector<Step> Steps;

// barrier and parity of what is told of tile t
static Step scores(Kind k, int t) { return {k, S0 + tile_bar(t), tile_parity(t), t / kTileBars + 1}; }
static Step weights(Kind k, int t) { return {k, P0 + tile_bar(t), tile_parity(t), t / kTileBars + 1}; }

static Steps issuer(const std::vector<int>& pieces) {
  Steps s;
  int t0 = 0;
  for (int p = 0; p < (int)pieces.size(); ++p) {
    s.push_back({WAIT, Q, p & 1u, p + 1});
    s.push_back(scores(COMMIT, t0));
    for (int i = 0; i < pieces[p]; ++i) {
      const int t = t0 + i;
      if (i + 1 < pieces[p]) s.push_back(scores(COMMIT, t + 1));
      s.push_back(weights(WAIT, t));
      if (i == 0 && p > 0) s.push_back({WAIT, DRAINED, (p - 1) & 1u, p});
      s.push_back({COMMIT, O, 0, 0});
    }
    s.push_back({COMMIT, FIN, 0, 0});
    t0 += pieces[p];
  }
  return s;
}
static Steps softmax(const std::vector<int>& pieces) {
  Steps s;
  int t0 = 0;
  s.push_back({ARRIVE, Q, 0, 0});
  for (int p = 0; p < (int)pieces.size(); ++p) {
    for (int i = 0; i < pieces[p]; ++i) {
      const int t = t0 + i;
      s.push_back(scores(WAIT, t));
      if (i > 0) s.push_back({MAY_WAIT, O, (t - 1) & 1u, t});  // only where the maximum moves
      s.push_back(weights(ARRIVE, t));
    }
    if (p + 1 < (int)pieces.size()) s.push_back({ARRIVE, Q, 0, 0});
    s.push_back({WAIT, FIN, p & 1u, p + 1});
    s.push_back({ARRIVE, DRAINED, 0, 0});
    t0 += pieces[p];
  }
  return s;
}

static int run(const std::vector<int>& pieces) {
  const Steps a = issuer(pieces), b = softmax(pieces);
  // (issuer's place, softmax's place, products complete): the rest follows from these
  typedef std::tuple<int, int, int> State;
  std::set<State> seen;
  std::vector<State> open = {State(0, 0, 0)};
  while (!open.empty()) {
    const State st = open.back();
    open.pop_back();
    if (!seen.insert(st).second) continue;
    const int ia = std::get<0>(st), ib = std::get<1>(st), done = std::get<2>(st);
    int phases[BARS] = {}, commits = 0;
    for (int i = 0; i < ia; ++i)
      if (a[i].kind == COMMIT && commits++ < done) ++phases[a[i].bar];
    for (int i = 0; i < ib; ++i)
      if (b[i].kind == ARRIVE) ++phases[b[i].bar];
    bool moved = false;
    auto step = [&](const Step& s, State next) {
      // a wait passes when the phase in progress has the other parity
      if (s.kind == WAIT || s.kind == MAY_WAIT) {
        const bool passes = (phases[s.bar] & 1u) != s.parity;
        if (passes && phases[s.bar] < s.phase) {
          printf("a wait passes early: barrier %d, phase %d of %d\n", s.bar, phases[s.bar], s.phase);
          return false;
        }
        if (!passes && s.kind == WAIT) return true;
        if (!passes) {  // whether it is waited for or not: both
          moved = true;
          open.push_back(next);
          return true;
        }
      }
      moved = true;
      open.push_back(next);
      return true;
    };
    if (ia < (int)a.size() && !step(a[ia], State(ia + 1, ib, done))) return 1;
    if (ib < (int)b.size() && !step(b[ib], State(ia, ib + 1, done))) return 1;
    if (done < commits) {
      moved = true;
      open.push_back(State(ia, ib, done + 1));
    }
    // a place where the optional wait is taken must not be a dead end either
    if (ib < (int)b.size() && b[ib].kind == MAY_WAIT && (phases[b[ib].bar] & 1u) == b[ib].parity &&
        phases[b[ib].bar] >= b[ib].phase) {
      printf("a phase has gone by unseen: barrier %d\n", b[ib].bar);
      return 1;
    }
    if (!moved && !(ia == (int)a.size() && ib == (int)b.size())) {
      printf("nothing moves: issuer at %d of %zu, softmax at %d of %zu, products %d of %d\n", ia, a.size(),
             ib, b.size(), done, commits);
      return 1;
    }
  }
  return 0;
}

int main() {
  for (const auto& p : std::vector<std::vector<int>>{{1}, {2}, {3}, {7}, {1, 1}, {1, 2, 3}, {4, 1, 1, 5}, {2, 2, 2}})
    if (run(p)) return 1;
  puts("ok");
  return 0;
}
"""


def test_every_order_of_steps_ends(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "bars.cpp", tmp_path / "bars"
    src.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout
