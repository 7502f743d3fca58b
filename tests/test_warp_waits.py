"""The bounded waits of whole warps, on the CPU: 32 threads stand for the lanes of
a warp, each with a barrier and a clock of its own, as lanes that poll one after
another see them.  Whatever they see, all lanes must get the same answer."""

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_attention_scores_b200", "csrc")

HARNESS = r"""
#include <atomic>
#include <condition_variable>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <random>
#include <thread>
#include <vector>
#define __device__
#define __forceinline__ inline

// a vote: every lane arrives with its value and leaves with everybody's
struct Vote {
  std::mutex m;
  std::condition_variable cv;
  int in = 0, round = 0;
  bool all = true, any = false, out_all = false, out_any = false;
  void cast(bool v, bool *o_all, bool *o_any) {
    std::unique_lock<std::mutex> lock(m);
    all = all && v;
    any = any || v;
    const int mine = round;
    if (++in == 32) {
      out_all = all;
      out_any = any;
      all = true;
      any = false;
      in = 0;
      ++round;
      cv.notify_all();
    } else {
      cv.wait(lock, [&] { return round != mine; });
    }
    *o_all = out_all;
    *o_any = out_any;
  }
};
static Vote *vote;
struct Lane {
  long tries = 0, completes = 0;  // the try from which on the barrier is seen complete
  long fails = 0;                 // the try at which another role's failure appears
  uint64_t now = 0, tick = 1;
  volatile uint32_t *failed = nullptr;
};
static thread_local Lane *me;
static int __all_sync(unsigned, bool v) { bool a, b; vote->cast(v, &a, &b); return a; }
static int __any_sync(unsigned, bool v) { bool a, b; vote->cast(v, &a, &b); return b; }
namespace dsa {
static bool mbar_try_wait(uint64_t *, uint32_t) {
  if (me->fails && me->tries >= me->fails) *me->failed = 1u;
  return me->tries++ >= me->completes;
}
static uint64_t global_timer_ns() { return me->now += me->tick; }
}
#include "warp_wait.cuh"

int main(int argc, char **argv) {
  std::mt19937 rng(7);
  auto pick = [&](long lo, long hi) { return std::uniform_int_distribution<long>(lo, hi)(rng); };
  int parted = 0, gave_up = 0, passed = 0;
  for (int run = 0; run < 75; ++run) {
    Vote v;
    vote = &v;
    volatile uint32_t failed = 0;
    std::vector<Lane> lane(32);
    const int kind = run % 3;
    for (auto &l : lane) {
      l.failed = &failed;
      l.completes = kind == 0 ? pick(0, 200) : pick(0, 20000);   // 0: always in time
      l.tick = kind == 1 ? pick(1, 200) : 1;                      // 1: some lanes' limits run out
      l.fails = kind == 2 ? pick(1, 400) : 0;                     // 2: another role fails
    }
    int answer[32];
    std::vector<std::thread> t;
    for (int i = 0; i < 32; ++i)
      t.emplace_back([&, i] {
        me = &lane[i];
        answer[i] = dsa::wait_or_fail(nullptr, 0u, kind == 0 ? 1000000u : 1000u, &failed);
      });
    for (auto &x : t) x.join();
    bool same = true;
    for (int i = 1; i < 32; ++i) same = same && answer[i] == answer[0];
    parted += !same;
    passed += answer[0] != 0;
    gave_up += answer[0] == 0;
    if (kind == 0 && !answer[0]) return std::printf("a wait that completes gave up\n"), 1;
    if (!answer[0] && !failed) return std::printf("gave up without saying so\n"), 1;
  }
  std::printf("parted %d, passed %d, gave up %d\n", parted, passed, gave_up);
  return parted != 0 || passed < 25 || gave_up < 25;
}
"""


@pytest.mark.parametrize("source", ["warp_wait.cuh"])
def test_all_lanes_get_the_same_answer(tmp_path, source):
    (tmp_path / "harness.cpp").write_text(HARNESS.replace("warp_wait.cuh", source))
    exe = tmp_path / "harness"
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-Wno-unknown-pragmas", "-I", CSRC,
                    str(tmp_path / "harness.cpp"), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout


@pytest.mark.parametrize("name", ["mass.cu", "mla4.cu"])
def test_whole_warps_wait_by_vote(name):
    """Outside the one thread that stalls for a test and the drain before a barrier of
    the whole CTA, every wait is the voting one, and no lane branches on a failure
    it has read by itself around what is for whole warps."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    waits = re.findall(r"mbar_wait\((\w+)", text)
    assert set(waits) <= {"bar_stall", "bar_drain"}, waits
    assert not re.search(r"mbar_try_wait", text)
    assert not re.search(r"if \(\*failed\)", text)
    assert not re.search(r"&& !\*failed\) publish", text)


def test_the_pipelined_bf16_and_e4m3_kernel_waits_by_vote_too():
    """Its MMA issuer is one thread with a wait of its own; the other roles are whole warps."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "mla.cu")).read())
    body = text[text.index("void __launch_bounds__(kPipeThreads, 1)"):]
    issue = body.index("else if (lane == 0) {")
    assert not re.search(r"pipe_wait|mbar_try_wait|mbar_wait\((?!bar_stall)", body[:issue])
    assert not re.search(r"if \(!?\*failed", body[:issue])
    assert len(re.findall(r"wait_or_fail\(", body[:issue])) == 5
