// Model of the chunk attention's operand ring over a pair of CTAs, on random schedules and stopped
// at a random moment: two loaders, loads that land late and in any order, the MMA warp that frees
// a slot, and the leader's barriers (arrivals and bytes).  After the stop, the leader follows
// kvk_chunk_stop.cuh.  Checked: its waits all end once the loads in flight have landed, and when
// they have ended no load is in flight (so that either CTA's memory may go).  Built and run by
// tests/test_chunk_stop_host.py; prints "ok <stops with loads in flight>" or the first failure.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "kvk_chunk_stop.cuh"

struct Barrier {
  int phase = 0, pending = 1;
  long tx = 0;
  void settle() {
    if (pending == 0 && tx == 0) {
      ++phase;
      pending = 1;
    }
  }
  void arrive_expect(long bytes) {
    tx += bytes;
    --pending;
    settle();
  }
  void complete(long bytes) {
    tx -= bytes;
    settle();
  }
  bool done(uint32_t parity) const { return (uint32_t)(phase & 1) != parity; }   // test_wait.parity
};
struct Load {
  int slot, rank;
  long bytes;
};

int main() {
  std::mt19937 rng(7);
  auto pick = [&](int n) { return (int)(rng() % (unsigned)n); };
  long busy = 0, one_sided[2] = {0, 0};
  for (int trial = 0; trial < 200000; ++trial) {
    const int slots = 1 + pick(8), steps = 1 + pick(40);
    std::vector<Barrier> ready(slots);
    std::vector<int> freed(slots, 0);         // k_empty: uses of the slot that are over, both CTAs'
    std::vector<Load> fly;
    int issued[2] = {0, 0}, used = 0;
    bool stopped[2] = {false, false}, stop = false, used_stopped = false;
    auto bytes = [&](int i) { return 100L + 10 * (i % 3); };   // a CTA's half of a step
    const int at = pick(12 * steps + 4);
    for (int tick = 0;; ++tick) {
      if (tick == at) stop = true;
      const int who = pick(4);
      if (who < 2 && !stopped[who]) {
        const int i = issued[who], s = i % slots;
        if (i == steps) {
          stopped[who] = true;                // its part is over
        } else if (freed[s] >= i / slots) {   // (a wait that succeeds does not look at the stop)
          if (who == 0) ready[s].arrive_expect(2 * bytes(i));
          for (int part = 0; part < 2; ++part) fly.push_back({s, who, bytes(i) / 2});
          ++issued[who];
        } else if (stop) {
          stopped[who] = true;
        }
      } else if (who == 2 && !used_stopped) {
        const int s = used % slots;
        if (used == steps) {
          used_stopped = true;
        } else if (ready[s].done((uint32_t)(used / slots) & 1u)) {
          for (const Load& l : fly)
            if (l.slot == s) return printf("trial %d: step %d used while a load is in flight\n", trial, used), 1;
          ++freed[s];
          ++used;
        } else if (stop) {
          used_stopped = true;
        }
      } else if (who == 3 && !fly.empty()) {
        const int k = pick((int)fly.size());
        const Load l = fly[k];
        fly.erase(fly.begin() + k);
        ready[l.slot].complete(l.bytes);
      }
      if (stopped[0] && stopped[1] && used_stopped) break;
      if (tick > 100000) return printf("trial %d: the model does not end\n", trial), 1;
    }
    if (!fly.empty()) ++busy;
    if (issued[0] != issued[1]) ++one_sided[issued[0] < issued[1]];
    // the stop: the leader's waits, with the loads landing meanwhile
    const int own = issued[0], peer = issued[1], top = own > peer ? own : peer;
    for (int i = kvk::chunk::stop_first(slots, own, peer); i < top; ++i) {
      const kvk::chunk::StopStep t = kvk::chunk::stop_step(i, slots, own, peer);
      if (t.arm) ready[t.slot].arrive_expect(bytes(i));
      if (t.complete) ready[t.slot].complete(bytes(i));
      while (!ready[t.slot].done(t.parity)) {
        if (fly.empty())
          return printf("trial %d: the wait for step %d (slots %d, issued %d and %d) never ends\n", trial,
                        i, slots, own, peer), 1;
        const int k = pick((int)fly.size());
        const Load l = fly[k];
        fly.erase(fly.begin() + k);
        ready[l.slot].complete(l.bytes);
      }
    }
    if (!fly.empty())
      return printf("trial %d: %zu loads in flight after the stop (slots %d, issued %d and %d)\n", trial,
                    fly.size(), slots, own, peer), 1;
  }
  if (!one_sided[0] || !one_sided[1]) return printf("no one-sided stops\n"), 1;
  printf("ok %ld\n", busy);
  return 0;
}
