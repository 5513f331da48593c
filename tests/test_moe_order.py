"""The order in which the expert layer's builder warps work and meet
(csrc/moe_order.h), run on the host: four threads for the four warps, whose waits
give up one by one in every combination.  All must leave together; a warp that
waits at a barrier for others that never come is a kernel that never ends."""
import os
import shutil
import subprocess

import pytest

from dense_gemm_tmem_gb300 import build

HARNESS = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>
#include <vector>
#include "moe_order.h"

// A barrier of four that also says whether all were ok, and whether it came at all.
struct Barrier {
  std::mutex m;
  std::condition_variable cv;
  int waiting = 0, turn = 0;
  bool all = true, result = true, stuck = false;
  bool meet(bool ok) {
    std::unique_lock<std::mutex> l(m);
    all = all && ok;
    const int mine = turn;
    if (++waiting == 4) {
      result = all;
      all = true;
      waiting = 0;
      ++turn;
      cv.notify_all();
      return result;
    }
    if (!cv.wait_for(l, std::chrono::milliseconds(500), [&] { return turn != mine || stuck; }) ||
        stuck) {
      stuck = true;
      cv.notify_all();
      return false;
    }
    return result;
  }
};

struct Case {
  int gave_up[2];  // warps whose waits give up in phase C, in phase D
  bool grid[2];    // whether the grid's barriers come
};

struct Warp {
  Barrier& b;
  const Case& c;
  int id, contents_run = 0, rows_run = 0, meetings = 0;
  bool contents(int phase) {
    ++contents_run;
    return !((c.gave_up[phase] >> id) & 1);
  }
  bool partials(bool ok) {
    ++meetings;
    return b.meet(ok && (id != 0 || c.grid[0]));
  }
  void rows() { ++rows_run; }
  bool rows_done() {
    ++meetings;
    return b.meet(id != 0 || c.grid[1]);
  }
};

int main() {
  int bad = 0;
  for (int first = 0; first < 16; ++first)
    for (int second = 0; second < 16; second += 5)
      for (int grid = 0; grid < 4; ++grid) {
        const Case c{{first, second}, {(grid & 1) != 0, (grid & 2) != 0}};
        Barrier b;
        std::vector<Warp> w;
        for (int i = 0; i < 4; ++i) w.push_back(Warp{b, c, i});
        std::vector<std::thread> t;
        for (int i = 0; i < 4; ++i) t.emplace_back([&, i] { dg::builder_run(w[i]); });
        for (auto& x : t) x.join();
        const bool on = first == 0 && c.grid[0], last = on && c.grid[1];
        for (int i = 0; i < 4; ++i)
          if (b.stuck || b.waiting != 0 || w[i].meetings != w[0].meetings ||
              w[i].rows_run != (on ? 1 : 0) || w[i].contents_run != (last ? 2 : 1)) {
            std::printf("first %d second %d grid %d: warp %d met %d times%s\n", first, second, grid,
                        i, w[i].meetings, b.stuck ? ", stuck" : "");
            ++bad;
            break;
          }
        if (bad > 3) return 1;
      }
  return bad != 0;
}
"""


def test_builder_warps_leave_together(tmp_path):
    cxx = os.environ.get("CXX", "g++")
    if shutil.which(cxx) is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "order.cpp", tmp_path / "order"
    src.write_text(HARNESS)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
