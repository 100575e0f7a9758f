"""The order in which a warpgroup of the block-scaled product leaves its tiles when bounded waits
give up, on the host: csrc/gemm_fp8_flow.cuh compiled with the C++ compiler, four threads in the
place of the four warps, waits that fail at every place, and barriers that report a thread which
never comes instead of waiting for good."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hybrid_masked_attention_b200", "csrc")

SOURCE = r"""
#include <atomic>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <mutex>
#include <set>
#include <thread>
#include <vector>

#include "gemm_fp8_flow.cuh"

// A barrier of the four: returns the vote, or marks itself stuck when some warp has left for good.
struct Barrier {
  std::mutex m;
  std::condition_variable cv;
  int here = 0, gone = 0, round = 0;
  bool all = true, result = true, stuck = false;
  bool arrive(bool ok) {
    std::unique_lock<std::mutex> l(m);
    all = all && ok;
    const int r = round;
    if (++here == 4) {
      result = all; all = true; here = 0; ++round;
      cv.notify_all();
      return result;
    }
    cv.wait(l, [&] { return round != r || gone > 0; });
    if (round != r) return result;
    stuck = true;  // a warp has left and never comes: on the device this waits for good
    return false;
  }
  void leave() {
    std::lock_guard<std::mutex> l(m);
    ++gone;
    cv.notify_all();
  }
};

// Waits of a warp are numbered in its own order; those in `fails` give up, and raise the flag.  Once it
// is up, a wait may still find its phase complete (`lucky`) or give up at once.
struct Warp {
  Barrier* b;
  std::atomic<int>* flag;
  std::set<int> fails;
  int waits = 0, stores = 0, tiles, blocks;
  bool residual, lucky;
  bool wait() {
    if (fails.count(waits++)) *flag = 1;
    else if (lucky || *flag == 0) return true;
    return false;
  }
};

template <bool kVote, bool kAhead>
void now(Warp& w) {
  auto scale = [&] { w.wait(); };
  auto begin = [&](int) {};
  auto blocks = [&](int t) {
    for (int k = 0; k < w.blocks; ++k) {
      if (!w.wait()) return;
      if (k + 1 < w.blocks || (kAhead && t + 1 < w.tiles)) scale();
    }
  };
  auto vote = [&] { return kVote ? w.b->arrive(*w.flag == 0) : *w.flag == 0; };
  auto finish = [&](int) {
    if (w.residual) w.wait();
    if (kVote) w.b->arrive(true);
    ++w.stores;
  };
  mtfm::epilogue_tiles<kAhead>(0, w.tiles, 1, scale, begin, blocks, vote, finish, [] {});
}

// The order before: a warp whose wait gave up outside of the blocks left by itself.
template <bool kVote, bool kAhead>
void before(Warp& w) {
  bool ok = true;
  if (kAhead) ok = w.wait();
  for (int t = 0; ok && t < w.tiles; ++t) {
    if (!kAhead) ok = w.wait();
    if (!ok) break;
    for (int k = 0; k < w.blocks; ++k) {
      if (!w.wait()) { ok = false; break; }
      if (k + 1 < w.blocks || (kAhead && t + 1 < w.tiles)) ok = w.wait();
    }
    if (kVote) ok = w.b->arrive(ok);
    if (!ok) break;
    if (w.residual) { ok = w.wait(); w.b->arrive(true); }
    else if (kVote) w.b->arrive(true);
    w.stores += ok;
  }
}

// stuck barriers over all runs; -1 where the warps of a run did not agree on the tiles they stored
template <class F>
int runs(F flow, bool vote, bool residual) {
  int stuck = 0;
  for (int tiles = 0; tiles <= 3; ++tiles)
    for (int blocks = 1; blocks <= 3; ++blocks)
      for (int who = 0; who < 16; ++who)  // which warps fail
        for (int at = 0; at < 24; ++at) {
          Barrier b;
          std::atomic<int> flag{0};
          Warp w[4];
          std::vector<std::thread> th;
          for (int i = 0; i < 4; ++i) {
            w[i].b = &b, w[i].flag = &flag, w[i].lucky = at + i & 1, w[i].tiles = tiles, w[i].blocks = blocks, w[i].residual = residual;
            if (who >> i & 1) w[i].fails = {at + i % 2, at + 7};
          }
          for (int i = 0; i < 4; ++i) th.emplace_back([&, i] { flow(w[i]); b.leave(); });
          for (auto& t : th) t.join();
          stuck += b.stuck;
          if (vote && !b.stuck)
            for (int i = 1; i < 4; ++i)
              if (w[i].stores != w[0].stores) return -1;
          if (who == 0 && w[0].stores != tiles) return -1;
        }
  return stuck;
}

int main() {
  // staged outputs (votes), with and without the scale fetched ahead; with a residual's wait; direct outputs
  std::printf("%d %d %d %d ", runs(now<true, true>, true, false), runs(now<true, false>, true, false),
              runs(now<true, false>, true, true), runs(now<false, true>, false, false));
  std::printf("%d\n", runs(now<false, false>, false, false));
  std::printf("%d %d %d\n", runs(before<true, true>, false, false), runs(before<true, false>, false, false),
              runs(before<true, false>, false, true));
}
"""


def test_no_warp_leaves_a_barrier_alone(tmp_path):
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "flow.cpp", tmp_path / "flow"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=300).stdout.split("\n")
    assert [int(v) for v in out[0].split()] == [0, 0, 0, 0, 0]
    # the order that let a warp leave by itself is found out in each staged form
    assert all(int(v) > 0 for v in out[1].split())


def test_kernel_goes_through_the_tested_order():
    """The kernel's tile loop is the tested function, and its unbounded barriers stand in its parts alone."""
    text = open(os.path.join(CSRC, "gemm_fp8.cu")).read()
    epilogue = text[text.index("scaling and epilogue"):text.index("every store has completed before the CTA leaves")]
    assert epilogue.count("epilogue_tiles<") == 1
    assert "for (int t =" not in epilogue and "break;" not in epilogue
