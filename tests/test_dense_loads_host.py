"""The books that a loader of the dense attention keeps of its copies, on the CPU:
when a wait runs out, at any claim and at any state of the ring, the drain waits for
every copy of the loader that is still on its way."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_long_fp8_b200", "csrc")

MODEL = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "dense_loads.cuh"

// The ring as the two loaders see it: 8 slots; entries in the order S(0), S(1),
// V(0), S(2), V(1), ..., five per S, four per V, the last V's second half by `tail`, one entry at a time.
static const unsigned RING = 8;
struct Copy { unsigned entry; int loader; bool tail; };
static unsigned rnd() { return static_cast<unsigned>(rand()) >> 4; }

int main(int argc, char** argv) {
  srand(atoi(argv[1]));
  long waited = 0, failed_in_flight = 0;
  for (int trial = 0; trial < 20000; ++trial) {
    const int n = 1 + rnd() % 6;
    std::vector<std::vector<unsigned>> mine(2);
    std::vector<char> by_tail;
    unsigned e = 0;
    for (int i = 0; i <= n; ++i) {
      if (i < n) for (int t = 0; t < 5; ++t) { mine[0].push_back(e++); by_tail.push_back(0); }
      if (i > 0) for (int t = 0; t < 4; ++t) { mine[1].push_back(e++); by_tail.push_back(i == n && t >= 2); }
    }
    dsa::DenseLoads<RING> loads[2];
    size_t next[2] = {0, 0};
    std::vector<Copy> flying;                  // issued, not landed
    std::vector<unsigned> done(RING, 0);       // uses of a slot that its full barrier has completed
    std::vector<unsigned> read(RING, 0);       // uses that the MMAs have read
    unsigned mma = 0;                          // next entry that the MMAs read
    auto land = [&](size_t i) {
      if (!flying[i].tail) ++done[flying[i].entry % RING];
      flying.erase(flying.begin() + i);
    };
    const unsigned stop = rnd() % (2 * e + 1); // steps until a wait runs out
    for (unsigned step = 0;; ++step) {
      const int who = rnd() & 1;
      const bool out = step >= stop;
      if (!out && !flying.empty() && (rnd() & 1)) {
        const size_t i = rnd() % flying.size();
        if (!flying[i].tail) land(i);
        continue;
      }
      if (!out && (rnd() & 1)) {
        if (mma < e && done[mma % RING] > mma / RING) { ++read[mma % RING]; ++mma; }
        continue;
      }
      bool lost = false;
      if (next[who] < mine[who].size()) {
        const unsigned en = mine[who][next[who]];
        unsigned slot = 99;
        const bool got = loads[who].claim(en, slot, [&](unsigned s, unsigned use) { return read[s] > use; });
        if (slot != en % RING) { printf("slot\n"); return 1; }
        if (got) {
          ++next[who];
          flying.push_back({en, who, by_tail[en] != 0});
          if (by_tail[en]) {
            loads[who].by_tail(slot);
            if (out) {                         // the wait for `tail` runs out
              lost = true;
            } else {                           // it lands; then the loader arrives itself
              land(flying.size() - 1);
              ++done[slot];
              loads[who].tail_landed();
            }
          }
        } else if (out) {
          lost = true;
        }
      } else if (out) {
        break;
      }
      if (!lost) {
        if (out && step > stop + 400) { printf("no end\n"); return 1; }
        continue;
      }
      for (auto& c : flying) failed_in_flight += c.loader == who;
      loads[who].drain(
          [&](unsigned s, unsigned parity) {
            if ((done[s] & 1) != parity) return;           // the phase is complete: returns at once
            for (size_t i = 0; i < flying.size(); ++i)
              if (flying[i].entry % RING == s && !flying[i].tail) { land(i); ++waited; break; }
          },
          [&] {
            for (size_t i = 0; i < flying.size(); ++i)
              if (flying[i].tail && flying[i].loader == who) { land(i--); ++waited; }
          });
      for (auto& c : flying)
        if (c.loader == who) { printf("trial %d: entry %u of loader %d is still on its way\n", trial, c.entry, who); return 1; }
      break;
    }
  }
  printf("%ld waited for of %ld\n", waited, failed_in_flight);
  return waited > 1000 && failed_in_flight > 1000 ? 0 : 1;
}
"""


def test_drain_waits_for_every_copy(tmp_path):
    src, exe = tmp_path / "model.cpp", tmp_path / "model"
    src.write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-x", "c++", f"-I{CSRC}", str(src), "-o",
                    str(exe)], check=True)
    for seed in ("1", "2"):
        r = subprocess.run([str(exe), seed], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout
