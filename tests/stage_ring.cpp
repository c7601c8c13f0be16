// Runs the ring of csrc/stage_ring.h among host threads: a filling thread, four
// readers of every stage, and copies that arrive late or not before a wait has
// run out.  Exits 0 when no stage is filled while a copy into it is under way,
// no barrier is armed in a phase that is not over, and no copy is under way when
// the filling thread ends.
//
//   stage_ring <fills> <late> <delay ms> <reader limit ms> <filler limit ms>
//
// `late`: the fill whose copy takes `delay`; all others take none.
//
//   stage_ring turns <stages> <takers> <late> <delay ms>
//
// Readers that take the fills in turn, by parity, while copies arrive in order:
// exits 0 when each found its fill's data, 1 when one was a round ahead; 4 when
// turns_are_safe() says otherwise.
#include <atomic>
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <string>
#include <thread>
#include <vector>

#include "stage_ring.h"

using namespace std::chrono;

namespace {

constexpr int kStages = 4, kReaders = 4;

// A barrier that counts arrivals and bytes, as the device's do.
struct Barrier {
  std::mutex m;
  std::condition_variable c;
  int count = 0, pending = 0, bytes = 0;
  uint32_t phase = 0;  // completed ones
  bool overrun = false;

  void init(int n) { count = pending = n; }
  void settle() {
    if (pending == 0 && bytes == 0) {
      pending = count;
      ++phase;
      c.notify_all();
    }
  }
  void arrive(int expect = 0) {
    std::lock_guard<std::mutex> l(m);
    if (pending == 0) overrun = true;  // more arrivals than the phase has
    else --pending;
    bytes += expect;
    settle();
  }
  void complete(int n) {
    std::lock_guard<std::mutex> l(m);
    bytes -= n;
    settle();
  }
  bool wait(uint32_t parity, milliseconds limit) {
    std::unique_lock<std::mutex> l(m);
    return c.wait_for(l, limit, [&] { return (phase & 1) != parity; });
  }
};

struct Block {
  Barrier full[kStages], free[kStages];
  std::atomic<int> under_way[kStages] = {};
  std::atomic<int> flag{0};
  std::atomic<bool> over{false};
};

struct Ops {
  Block& b;
  milliseconds limit, drain_limit;
  bool wait_full(uint32_t s, uint32_t parity) { return b.full[s].wait(parity, drain_limit); }
  bool wait_free(uint32_t s, uint32_t parity) { return b.free[s].wait(parity, limit); }
  bool raised() { return b.flag.load() != 0; }
  void raise() { b.flag.store(1); }
  bool any(bool v) { return v; }
};

int turns(int stages, int takers, int late, milliseconds delay) {
  const int fills = 12 * stages;
  std::vector<Barrier> full(stages), free(stages);
  std::vector<std::atomic<int>> data(stages);
  for (int i = 0; i < stages; ++i) full[i].init(1), free[i].init(1), data[i] = -1;
  std::atomic<bool> wrong{false};
  std::thread filler([&] {
    for (int i = 0; i < fills && !wrong; ++i) {
      const int s = i % stages;
      if (i >= stages) free[s].wait((i / stages - 1) & 1, seconds(10));
      if (i == late) std::this_thread::sleep_for(delay);
      data[s] = i;
      full[s].arrive();
    }
  });
  std::vector<std::thread> readers;
  for (int w = 0; w < takers; ++w)
    readers.emplace_back([&, w] {
      for (int u = w; u < fills && !wrong; u += takers) {
        const int s = u % stages;
        for (int tries = 0; tries < 1000 && !wrong && !full[s].wait((u / stages) & 1, milliseconds(20)); ++tries) {
        }
        if (data[s] != u) wrong = true;
        free[s].arrive();
      }
    });
  filler.join();
  for (auto& t : readers) t.join();
  return wrong ? 1 : 0;
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 6) return 2;
  if (std::string(argv[1]) == "turns") {
    const int wrong = turns(atoi(argv[2]), atoi(argv[3]), atoi(argv[4]), milliseconds(atoi(argv[5])));
    const bool safe = qlin::ring::turns_are_safe(atoi(argv[2]), atoi(argv[3]));
    return wrong && safe ? 4 : wrong;
  }
  const int fills = atoi(argv[1]), late = atoi(argv[2]);
  const milliseconds delay(atoi(argv[3])), reader_limit(atoi(argv[4])), filler_limit(atoi(argv[5]));
  Block b;
  for (int i = 0; i < kStages; ++i) b.full[i].init(1), b.free[i].init(kReaders);
  std::vector<std::thread> copies, readers;
  int issued = 0;

  std::thread filler([&] {
    Ops ops{b, filler_limit, delay + seconds(10)};
    qlin::ring::Filler<kStages> fill;
    for (int i = 0; i < fills; ++i) {
      if (!fill.wait(ops)) continue;
      const uint32_t s = fill.stage();
      if (b.under_way[s].fetch_add(1) != 0) b.over = true;
      b.full[s].arrive(16);
      ++issued;
      copies.emplace_back([&, s, i] {
        if (i == late) std::this_thread::sleep_for(delay);
        b.under_way[s].fetch_sub(1);
        b.full[s].complete(16);
      });
      ++fill.filled;
    }
    fill.drain(ops);
    for (int i = 0; i < kStages; ++i)
      if (b.under_way[i].load() != 0) b.over = true;
  });
  for (int r = 0; r < kReaders; ++r)
    readers.emplace_back([&, r] {
      Ops ops{b, reader_limit, reader_limit};
      bool ran_out = false;
      for (int i = 0; i < fills; ++i) {
        const uint32_t s = i % kStages;
        qlin::ring::wait_or_raise(ops, ran_out, [&] { return b.full[s].wait((i / kStages) & 1, reader_limit); });
        if (r == 1 && i % 3 == 0) std::this_thread::sleep_for(microseconds(200));  // readers drift apart
        b.free[s].arrive();
      }
    });
  filler.join();
  for (auto& t : readers) t.join();
  for (auto& t : copies) t.join();
  for (int i = 0; i < kStages; ++i)
    if (b.full[i].overrun) b.over = true;
  printf("issued %d of %d, flag %d\n", issued, fills, b.flag.load());
  if (b.over) return 1;
  const bool calm = delay < reader_limit && delay < filler_limit;
  return calm && (issued != fills || b.flag.load() != 0) ? 3 : 0;
}
