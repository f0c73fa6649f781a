"""Host checks of the packed-token operators where a GPU run could not show the
mistake, or could not run it safely."""
import ctypes
import os
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "state_space_model_scan_amd", "csrc")

RUNS = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <vector>
#include "conv_runs.h"
using namespace ssm;
typedef std::vector<int64_t> Edges;

// a run that computes its own tokens and no others
template <typename Edge, typename Piece>
void own_tokens(const Edge &edge, int64_t nseq, int64_t total, int64_t t0, int n, int64_t s, Piece &&piece) {
  for (int from = 0; from < n;) {
    while (t0 + from >= edge(s + 1) && s + 1 < nseq) ++s;
    const int64_t left = edge(s + 1) - t0;
    const int to = s + 1 < nseq && left < n ? (int)left : n;
    piece(s, from, to, t0 + from - first_token(edge, s), edge(s + 1));
    from = to;
  }
}

// every token computed once, at its place, and no ring of two runs; NULL or what is wrong
template <bool OWN>
const char *check(const Edges &cu, int run) {
  const int64_t nseq = cu.size() - 1, total = cu.back();
  auto edge = [&](int64_t i) { return cu.at(i); };
  std::vector<int> done(total, 0);
  std::map<int64_t, std::set<int64_t>> users;   // sequence -> runs that read or write its ring
  const char *bad = nullptr;
  for (int64_t t0 = 0; t0 < total; t0 += run) {
    int64_t s0 = 0;
    for (int64_t s = 0; s < nseq; ++s) if (cu[s] <= t0) s0 = s;
    auto piece = [&](int64_t s, int from, int to, int64_t pos, int64_t end) {
      if (from >= to || to > run + kTaps - 2 || t0 + to > total) { bad = "a piece's bounds"; return; }
      if (pos != t0 + from - cu[s] || end != cu[s + 1] || t0 + to > end) { bad = "a piece's place"; return; }
      for (int i = from; i < to; ++i) ++done[t0 + i];
      if (pos < kTaps - 1) users[s].insert(t0);
    };
    const int n = total - t0 < run ? (int)(total - t0) : run;
    if (OWN) own_tokens(edge, nseq, total, t0, n, s0, piece);
    else run_pieces(edge, nseq, total, t0, n, s0, piece);
  }
  for (int v : done) if (v != 1) bad = "a token not computed once";
  for (auto &u : users) if (u.second.size() != 1) bad = "a ring of two runs";
  return bad;
}

int main() {
  std::mt19937 rng(5);
  long layouts = 0, shared = 0;
  for (int i = 0; i < 40000; ++i) {
    Edges cu = {0};
    const int nseq = 1 + rng() % 9, longest = (int[]){2, 5, 16, 60}[rng() % 4];
    for (int s = 0; s < nseq; ++s) cu.push_back(cu.back() + (rng() % 4 ? rng() % longest : rng() % 2));
    if (cu.back() == 0) continue;
    for (int run : {4, 12}) {
      ++layouts;
      if (const char *bad = check<false>(cu, run)) { printf("run %d: %s\n", run, bad); return 1; }
      if (check<true>(cu, run)) ++shared;
    }
  }
  if (shared < layouts / 20) { printf("the check sees too little: %ld of %ld\n", shared, layouts); return 1; }
  // edges out of order and out of range: every access stays inside the tokens
  for (int i = 0; i < 200000; ++i) {
    const int64_t total = 1 + rng() % 100, nseq = 1 + rng() % 6;
    Edges cu;
    for (int s = 0; s <= nseq; ++s) {
      const int kind = rng() % 8;
      cu.push_back(kind == 0 ? -(int64_t)(rng() % 20) : kind == 1 ? INT32_MAX : kind == 2 ? INT32_MIN : (int64_t)(rng() % 120));
    }
    const int run = rng() % 2 ? 4 : 12;
    for (int64_t t0 = 0; t0 < total; t0 += run) {
      bool bad = false;
      run_pieces([&](int64_t k) { return cu.at(k); }, nseq, total, t0, total - t0 < run ? (int)(total - t0) : run, rng() % nseq,
                 [&](int64_t s, int from, int to, int64_t pos, int64_t) {
        if (s < 0 || s >= nseq || from < 0 || from >= to || t0 + to > total) bad = true;
        for (int back = 1; back < kTaps; ++back) if (pos >= back && t0 + from - back < 0) bad = true;
      });
      // where all of a run and what it sees is read without a test
      const int64_t s = rng() % nseq;
      if (inside_one([&](int64_t k) { return cu.at(k); }, s, t0, t0 + run) && t0 - (kTaps - 1) < 0) bad = true;
      if (bad) { printf("edges out of order: outside the tokens\n"); return 1; }
    }
  }
  // far from the start, with edges at the ends of their type
  for (int64_t e : {(int64_t)INT32_MIN, (int64_t)-1, (int64_t)0, (int64_t)INT32_MAX - 3, (int64_t)INT32_MAX}) {
    const int64_t total = INT32_MAX, t0 = total / 12 * 12;
    const Edges cu = {e, e, e};
    bool bad = false;
    run_pieces([&](int64_t k) { return cu.at(k); }, 2, total, t0, (int)(total - t0), 1, [&](int64_t, int from, int to, int64_t, int64_t) {
      if (from < 0 || from >= to || t0 + to > total) bad = true;
    });
    if (bad) { printf("far edges: outside the tokens\n"); return 1; }
  }
  printf("%ld layouts, %ld of them shared between runs of their own tokens\n", layouts, shared);
  return 0;
}
"""


def _host_program(tmp_path, text):
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(text)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", f"-I{CSRC}", str(src), "-o", str(exe)], check=True, timeout=120)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout + res.stderr


SEEN = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include "conv_runs.h"
int main() {
  // a first edge below 0 stands for 0: the run of token 0 sees nothing before it
  for (int64_t first = -40; first <= 0; ++first) {
    const int64_t cu[2] = {first, 1000};
    auto edge = [&](int64_t k) { return cu[k]; };
    if (ssm::first_token(edge, 0) != 0) return 1;
    for (int t0 : {0, 1, 2, 3, 8, 32})
      if (ssm::inside_one(edge, 0, t0, t0 + 35) != (t0 >= 3)) { printf("token %d, edge %d\n", t0, (int)first); return 1; }
  }
  return 0;
}
"""


def test_a_first_edge_below_zero_stands_for_zero(tmp_path):
    _host_program(tmp_path, SEEN)


def test_one_run_reads_and_writes_a_ring(tmp_path):
    """The packed conv's runs, by the header the kernel uses: every token once,
    a sequence's ring read and written by one run only (which a split at the
    runs' ends is not), and nothing outside the tokens whatever the edges."""
    _host_program(tmp_path, RUNS)


def test_a_named_stream_is_the_calls_current_one(monkeypatch):
    """Every wrapper that takes a stream runs as a whole with it as the current
    one, whether it is passed by name or by place; without one nothing changes."""
    import contextlib
    import inspect
    import torch
    from state_space_model_scan_amd import binding
    entered = []

    @contextlib.contextmanager
    def stream(s):
        entered.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "stream", stream)
    names = [n for n, f in vars(binding).items() if inspect.isfunction(f) and f.__module__ == binding.__name__ and
             "stream" in inspect.signature(f).parameters and not n.startswith("_")]
    packed = {"causal_conv1d_varlen_fwd", "causal_conv1d_varlen_bwd", "ssd_varlen_fwd", "ssd_varlen_bwd", "conv1d_ssd_update"}
    assert packed < set(names) and len(names) == 18   # (those do it in C++)
    for name in sorted(set(names) - packed):
        f = getattr(binding, name)
        at = list(inspect.signature(f).parameters).index("stream")
        for args, kw in (((None,) * at, dict(stream="s")), ((None,) * at + ("s",), {}), ((None,) * at, {})):
            entered.clear()
            try:
                f(*args, **kw)
            except (AttributeError, TypeError, ValueError):
                pass   # (no tensors)
            assert entered == (["s"] if kw or len(args) > at else []), (name, args, kw)


@pytest.mark.parametrize("given", ["codes", "scales"])
def test_checkpoints_without_one_of_their_parts(given):
    """Refused: codes without scales were an access through nothing, scales
    without codes were dropped."""
    import torch
    from state_space_model_scan_amd import binding
    bf, T, h, n = torch.bfloat16, 70, 2, 32
    codes = torch.zeros(binding.ssd_checkpoint_slots(T, 1), h, 64, n, dtype=torch.int8)
    pair = (codes, None) if given == "codes" else (None, torch.ones(codes.shape[:3]))
    x, dt, B = torch.zeros(T, h, 64, dtype=bf), torch.zeros(T, h, dtype=bf), torch.zeros(T, 1, n, dtype=bf)
    with pytest.raises(ValueError, match="codes and their scales"):
        binding.ssd_varlen_fwd(x, dt, -torch.ones(h), B, B, torch.tensor([0, T], dtype=torch.int32), T, checkpoints=pair)
    with pytest.raises((ValueError, TypeError)):
        binding.ssd_varlen_bwd(x, dt, -torch.ones(h), B, B, torch.tensor([0, T], dtype=torch.int32), T, x, pair)


def test_weights_at_any_address():
    from state_space_model_scan_amd import _lib
    from tests.test_varlen_cpu import FAKE, _step, _st
    assert _st("conv1d_ssd_update", _step(conv_weight=FAKE + 4)) == _lib.SSM_OK


def test_grids_that_the_device_cannot_count_are_refused():
    """A launch has less than 2^32 threads in x: refused before anything is
    launched, with the shape's status and not the runtime's."""
    from state_space_model_scan_amd import _lib
    from tests.test_varlen_cpu import _conv, _scan, _scan_bwd

    def st(name, a):
        return getattr(_lib.lib(), name)(ctypes.byref(a), None)

    assert st("causal_conv1d_varlen_fwd", _conv(total=900_000_000)) == _lib.SSM_ERR_SHAPE
    many = dict(total=1 << 23, nseq=1 << 22, max_seqlen=4)   # 2^24 (sequence, head) pairs, 2^22 + 2^17 checkpoint entries
    assert st("ssd_varlen_fwd", _scan(**many)) == _lib.SSM_ERR_SHAPE
    assert st("ssd_varlen_bwd", _scan_bwd(many)) == _lib.SSM_ERR_SHAPE
    many.update(nseq=(1 << 22) - 1)
    assert st("ssd_varlen_bwd", _scan_bwd(many)) == _lib.SSM_ERR_WORKSPACE
