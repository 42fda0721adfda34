// Runs tree_unit() as a team of threads whose items wait and meet as the kernel's do, with waits
// that run out for any of the threads, and reports threads that are left at a barrier.
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <thread>
#include <vector>

#include "../kv_cache_quantization_x128_gb300/csrc/tree_unit.cuh"

constexpr int kThreads = 3;

struct Barrier {                 // of the whole team, answers the AND of what its threads bring
  std::mutex m;
  std::condition_variable cv;
  int in = 0, round = 0;
  bool all = true, answer = true, stuck = false;
  bool meet(bool mine) {
    std::unique_lock<std::mutex> lock(m);
    const int r = round;
    all = all && mine;
    if (++in == kThreads) {
      answer = all;
      all = true;
      in = 0;
      ++round;
      cv.notify_all();
      return answer;
    }
    if (!cv.wait_for(lock, std::chrono::seconds(20), [&] { return round != r; })) {
      stuck = true;              // the kernel would hang here
      return false;
    }
    return answer;
  }
};

// A thread of the team: an item agrees on what the waits before its softmax brought, and then waits
// for its second product, as TreeTeam::item does.
struct Thread {
  Barrier* bar;
  unsigned late;                 // bit i: the wait for item i's second product runs out
  unsigned early;                // bit i: the wait for its record or first product does
  bool ok = true;
  int done = 0;
  bool wait(unsigned mask, int i) const { return !((mask >> i) & 1u); }
  bool item(int i) {
    ok = wait(early, i) && ok;
    bar->meet(true);             // operands written
    if (!bar->meet(ok)) return ok = false;
    ok = wait(late, i) && ok;
    ++done;
    return true;
  }
  bool packed_item(int i) { return item(i); }
  bool fresh_item(int i) { return item(i); }
  bool unrotate() {
    bar->meet(true);
    return bar->meet(ok);
  }
  bool agreed() { return ok = bar->meet(ok); }
};

int main() {
  int bad = 0, runs = 0;
  for (int last = 0; last <= 2; ++last)
    for (int end = last; end <= last + 2; ++end)
      for (int item = 0; item < end; ++item)
        for (unsigned who = 0; who < (1u << kThreads); ++who)
          for (int when = 0; when < 2; ++when) {
            Barrier bar;
            std::vector<Thread> team;
            for (int t = 0; t < kThreads; ++t) {
              const unsigned mask = ((who >> t) & 1u) << item;
              team.push_back({&bar, when ? mask : 0u, when ? 0u : mask});
            }
            bool left[kThreads];
            std::vector<std::thread> threads;
            for (int t = 0; t < kThreads; ++t)
              threads.emplace_back([&, t] { left[t] = kvarn::tree_unit(team[t], 0, last, end); });
            for (auto& t : threads) t.join();
            ++runs;
            bool wrong = bar.stuck;
            for (int t = 0; t < kThreads; ++t) wrong = wrong || left[t] != (who == 0) || team[t].done != team[0].done;
            if (wrong && ++bad <= 5)
              std::printf("%d packed, %d fresh: a wait of item %d ran out for threads %x (%s)%s\n", last, end - last, item, who,
                          when ? "second product" : "before", bar.stuck ? ": left at a barrier" : "");
          }
  std::printf("%d runs, %d wrong\n", runs, bad);
  return bad ? 1 : 0;
}
