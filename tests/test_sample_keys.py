"""The sampler's keys (csrc/sample_keys.h), compiled for the host: every range of keys is the same
set of logits as the range of floats between its ends, so a bin's index never leaves the bins."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mtp_block_draft_gb300", "csrc")

PROGRAM = r"""
#include <math.h>
#include <stdio.h>
#include <algorithm>
#include <vector>
#include "sample_keys.h"

static int bad = 0;
#define CHECK(x, ...) do { if (!(x)) { if (bad++ < 5) { printf("%s: ", #x); printf(__VA_ARGS__); puts(""); } } } while (0)

// The k-th largest of v by repeated splits into 2^bits bins, as the kernels find it: members of a
// range by float comparison, bins by key.
static float kth(const std::vector<float>& v, uint32_t lo, uint32_t hi, unsigned want, int bits) {
  unsigned cnt = 0;
  for (float x : v) cnt += key_of(x) >= lo && key_of(x) <= hi;
  while (want != cnt && lo != hi) {
    const int shift = range_shift(lo, hi, bits);
    const float lf = logit_of(lo), hf = logit_of(hi);
    std::vector<unsigned> hist(1u << bits, 0u);
    for (float x : v)
      if (x >= lf && x <= hf) {
        const uint32_t place = (hi - key_of(x)) >> shift;
        CHECK(place < hist.size(), "logit %g range %g..%g place %u", x, lf, hf, place);
        if (place >= hist.size()) return NAN;
        ++hist[place];
      }
    unsigned f = 0, before = 0;
    while (f < hist.size() && before + hist[f] < want) before += hist[f++];
    CHECK(f < hist.size(), "want %u of %u in %g..%g", want, before, lf, hf);
    if (f >= hist.size()) return NAN;
    cnt = hist[f];
    want -= before;
    take_bin(lo, hi, shift, f);
  }
  // what is kept: everything from lo on
  float least = INFINITY;
  for (float x : v)
    if (x >= logit_of(lo)) least = std::min(least, x);
  return least;
}

int main() {
  // neighbours as floats are neighbours as keys
  std::vector<float> at = {-3.4028235e38f, -1e30f, -2.f, -1.f, -1.1754944e-38f, -1e-40f, -1.4e-45f, 0.f,
                           1.4e-45f, 1e-40f, 1.1754944e-38f, 1.f, 2.f, 1e30f};
  for (float a : at) {
    float x = a;
    for (int i = 0; i < 1000; ++i) {
      const float y = nextafterf(x, INFINITY);
      CHECK(key_of(y) - key_of(x) == 1u, "%g -> %g", x, y);
      CHECK(logit_of(key_of(x)) == x, "%g", x);
      x = y;
    }
  }
  CHECK(key_of(-0.f) == key_of(0.f), "zeros");
  CHECK(key_of(-INFINITY) == kMaskedKey && logit_of(kMaskedKey) == -INFINITY, "masked");
  CHECK(key_of(-3.4028235e38f) == kLowestKey, "lowest");
  // zeros beside the smallest negative numbers, ties, and both signs
  const std::vector<std::vector<float>> rows = {
      {1.9999999f, 0.f, 0.f, 0.f, -1e-40f, -2e-40f, -3e-40f},
      {1.f, 0.f, -0.f, -1.4e-45f, -1.4e-45f, -2.8e-45f, 1.4e-45f},
      {-0.f, -1.4e-45f, -1e-38f, -1.f, -2.f},
      {5.f, 5.f, 0.f, 0.f, -5.f, -5.f, -0.f, 1e-45f, -1e-45f},
      {0.f, 0.f, 0.f, 0.f}, {-1e-40f, -1e-40f, -2e-40f, 3.4028235e38f, -3.4028235e38f}};
  for (auto v : rows) {
    std::vector<float> s = v;
    std::sort(s.begin(), s.end(), [](float a, float b) { return a > b; });
    for (int bits : {9, 11})
      for (size_t a = 0; a < s.size(); ++a)       // ranges that end at any of the logits,
        for (size_t b = a; b < s.size(); ++b) {   // exactly or beside it
          unsigned n = 0;
          for (float x : v) n += x <= s[a] && x >= s[b];
          for (unsigned lo_off = 0; lo_off < 2; ++lo_off)
            for (unsigned hi_off = 0; hi_off < 2; ++hi_off)
              for (unsigned want = 1; want <= n; ++want) {
                const uint32_t lo = key_of(s[b]) - lo_off, hi = key_of(s[a]) + hi_off;
                std::vector<float> in;
                for (float x : s)
                  if (key_of(x) >= lo && key_of(x) <= hi) in.push_back(x);
                std::vector<float> members;
                for (float x : s)
                  if (x >= logit_of(lo) && x <= logit_of(hi)) members.push_back(x);
                CHECK(members == in, "keys and floats differ at %g..%g", s[b], s[a]);
                CHECK(kth(in, lo, hi, want, bits) == in[want - 1], "want %u from %g..%g", want, s[b], s[a]);
              }
        }
  }
  printf(bad ? "BAD %d\n" : "ok\n", bad);
  return bad != 0;
}
"""


def test_ranges_of_keys_are_ranges_of_logits(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "keys.cpp", tmp_path / "keys"
    src.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout
