"""The one- and two-token product's rings, on the host: every size's plan, and
the walk of the producer and the two groups over the slots."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_13_b200", "csrc")

PLANS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "rows_ring.cuh"
using namespace gptq::rows;

#define CHECK(x) do { if (!(x)) { std::printf("%s: G %d T %d in %d out %d ldw %lld sms %d\n", #x, G, T, in, out, \
                                              (long long)ldw, sms); std::exit(1); } } while (0)

// One block's batches.  The producer fills the slots of batch b in ring
// b % kGroups; group w waits for those of its batches.  mbarrier parity waits
// are safe if the waiting threads have waited for each of a slot's fills in turn
// and the parity is that of the fill.
void walk(int G, int T, int in, int out, int64_t ldw, int sms, const Plan& p) {
  const int R = kBatch / G, batches = (p.rows + R - 1) / R;
  std::vector<int> filled(kGroups * p.slots), waited(kGroups * p.slots);
  Cursor fill[kGroups], take[kGroups];
  for (auto& c : fill) c.phase = 1;
  for (int b = 0; b < batches; ++b) {
    const int ring = b % kGroups, left = p.rows - b * R, rows = left < R ? left : R;
    const int held = (rows + p.group - 1) / p.group;
    for (int i = 0; i < held; ++i, fill[ring].advance(1, p.slots)) {
      const int s = ring * p.slots + fill[ring].slot;
      CHECK(fill[ring].phase == ((filled[s] & 1) ^ 1));  // the fill before has been emptied
      ++filled[s];
    }
    for (int i = 0; i < held; ++i, take[ring].advance(1, p.slots)) {
      const int s = ring * p.slots + take[ring].slot;
      CHECK(take[ring].phase == (waited[s] & 1));
      ++waited[s];
      CHECK(waited[s] == filled[s]);
    }
  }
}

int main() {
  long long plans = 0;
  for (int G = 1; G <= 2; ++G)
    for (int T = 1; T <= 2; ++T)
      for (int in = 1; in <= kMaxSteps * kSlice; in += in < 64 || in > 12200 ? 1 : 61)
        for (int pad : {-1, 0, 16, 112, 128, 4096})
          for (int out : {1, 2, 147, 148, 149, 4096, 16384, 37888, 37889, 40000, 63048, 65535})
            for (int sms : {148, 132, 20}) {
              const int64_t ldw = pad < 0 ? 0 : (in + 15) / 16 * 16 + pad;
              const Plan p = plan(G, T, in, out, ldw, sms);
              CHECK(p.grid >= 1 && p.grid <= out && (sms < 148 || p.grid <= sms));
              CHECK((long long)p.rows * p.grid >= out && (p.rows - 1) * (long long)p.grid < out);
              CHECK(p.group >= 1 && kBatch / G % p.group == 0);
              const int batch = kBatch / G / p.group;
              CHECK(p.slots >= batch && p.slots <= kMaxSlots);
              CHECK(p.row_bytes >= in && p.row_bytes % 16 == 0);
              CHECK(!p.dense || p.row_bytes == ldw);
              CHECK(p.slot_bytes >= G * p.group * p.row_bytes && p.slot_bytes % 128 == 0);
              const int fixed = T * ((in + kSlice - 1) / kSlice) * kThreads * 16 + (G == 1 ? 12 : 16) * p.rows;
              CHECK(p.smem == fixed + kGroups * p.slots * p.slot_bytes);
              CHECK(p.smem + kStatic <= 232448);
              walk(G, T, in, out, ldw, sms, p);
              ++plans;
            }
  std::printf("%lld plans\n", plans);
}
"""


def test_every_plan_holds_and_each_group_waits_for_every_fill_of_its_slots(tmp_path):
    source = tmp_path / "plans.cpp"
    source.write_text(PLANS)
    exe = str(tmp_path / "plans")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-x", "c++", str(source), "-I", CSRC, "-o", exe],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout


def _early(slots, per_batch, batches, rings):
    """Waits (batch, slot) of a group that a fill it has not waited for can pass
    early: the slot's previous fill went to the other group."""
    last, early = {}, []
    at = [0] * rings
    for b in range(batches):
        ring = b % rings
        for _ in range(per_batch):
            s = (ring, at[ring] % slots)
            at[ring] += 1
            if last.get(s, b % 2) != b % 2:
                early.append((b, s))
            last[s] = b % 2
    return early


@pytest.mark.parametrize("slots,per_batch", [(7, 4), (9, 4), (13, 4), (5, 2)])
def test_a_ring_for_both_groups_would_let_a_wait_pass_early(slots, per_batch):
    assert _early(slots, per_batch, 40, 1)
    assert not _early(max(slots // 2, per_batch), per_batch, 40, 2)
