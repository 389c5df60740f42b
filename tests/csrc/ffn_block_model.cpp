// A model of the waits of the one-kernel feed-forward forward (csrc/ffn_block.cu), on the host: every warp is a list of waits, arrivals
// and asynchronous work; copies land and products finish after any time, in any order that the hardware allows (those that one warp
// issued in its order, all others in any). Barriers pass by parity, as the hardware's do, and the model knows which phase
// each wait means: a wait that passes before that phase is done is an error, and so is a schedule that stands still.
// Buffers, barriers and phases are those of csrc/ffn_schedule.cuh.
//
// usage: model channels shared seed runs   (channels: 128 or 256; shared: 1 for one barrier a buffer, whoever waits there)
// prints: early waits, runs that stood still, arrivals too many
#include <cstdio>
#include <cstdlib>
#include <deque>
#include <functional>
#include <memory>
#include <random>
#include <vector>

#include "ffn_schedule.cuh"

namespace {

struct Barrier {
  int count = 1, left = 1, phase = 0;
  void arrive() {
    if (--left == 0) {
      left = count;
      ++phase;
    }
  }
};

template <int NS, int NW, int XB, bool SHARED>
struct Model {
  using Order = triattn::ffn::BlockSchedule<NS, NW>;
  static constexpr int kSums = SHARED ? NS : Order::kSums;
  static int sums(int n) { return SHARED ? n % NS : Order::sums(n); }
  static int sums_phase(int n) { return SHARED ? n / NS : Order::sums_phase(n); }
  static constexpr int G = 2;  // warps of a group and CTA (8 in the kernel: no two of them wait for one another)

  struct Cta {  // what a CTA's barriers are
    Barrier xf[XB], xe[XB], wf[NW], we[NW], s[kSums], h[NS], of, oe;
  } cta[2];
  int tiles, blocks, early = 0;
  std::mt19937 rng;

  // A warp: steps that are done one after another, each as soon as its condition holds.
  struct Step {
    std::function<bool()> ready;
    std::function<void()> act;
  };
  struct Warp {
    std::deque<Step> steps;
    double speed = 1;
  };
  // Work in flight: queues whose members finish in order, each queue at its own pace.
  struct Flight {
    std::deque<std::function<void()>> work;
    double speed = 1;
  };
  std::vector<Warp> warps;
  std::vector<std::unique_ptr<Flight>> flights;

  Flight *flight() {
    flights.emplace_back(new Flight);
    flights.back()->speed = pace();
    return flights.back().get();
  }
  double pace() { return std::vector<double>{1, 1, 0.1, 0.01}[rng() % 4]; }

  // A wait for phase `n` of a barrier.
  void wait(Warp &w, Barrier &b, int n) {
    w.steps.push_back({[&b, n] { return (b.phase & 1) != (n & 1); }, [this, &b, n] { early += b.phase <= n; }});
  }
  void act(Warp &w, std::function<void()> f) {
    w.steps.push_back({[] { return true; }, f});
  }
  // A copy of one CTA's part: it lands whenever it likes.
  void copy(Warp &w, Barrier &b) {
    act(w, [this, &b] { flight()->work.push_back([&b] { b.arrive(); }); });
  }
  // The products that a warp has issued are done: both CTAs' barriers learn it, one after the other.
  void commit(Warp &w, Flight *f, Barrier &b0, Barrier &b1) {
    act(w, [f, &b0, &b1] {
      f->work.push_back([&b0] { b0.arrive(); });
      f->work.push_back([&b1] { b1.arrive(); });
    });
  }

  Model(int tiles, int blocks, unsigned seed) : tiles(tiles), blocks(blocks), rng(seed) {
    for (int r = 0; r < 2; ++r) {
      auto set = [](Barrier &b, int n) { b.count = b.left = n; };
      for (auto &b : cta[r].xf) set(b, 2);  // (both CTAs' copies)
      for (auto &b : cta[r].wf) set(b, 2);
      for (auto &b : cta[r].xe) set(b, 2);  // (both issuing warps)
      for (auto &b : cta[r].h) set(b, 2 * G);
      set(cta[r].oe, 4 * G);
    }
    warps.resize(2 + 3 + 4 * G);
    for (auto &w : warps) w.speed = pace();
    const int total = tiles * blocks;
    // both CTAs' copies: all count on the first one's barriers
    for (int r = 0; r < 2; ++r) {
      Warp &w = warps[r];
      int xs = 0, ws = 0;
      auto load_x = [&] {
        if (xs >= XB) wait(w, cta[r].xe[xs % XB], xs / XB - 1);
        copy(w, cta[0].xf[xs % XB]);
        ++xs;
      };
      load_x();
      for (int t = 0; t < tiles; ++t)
        for (int f = 0; f < blocks; ++f, ++ws) {
          if (ws >= NW) wait(w, cta[r].we[Order::slot(ws)], Order::slot_phase(ws - NW));
          copy(w, cta[0].wf[Order::slot(ws)]);
          if (t + 1 < tiles && f == (XB > 1 ? 0 : blocks - 1)) {
            load_x();
          }
        }
    }
    // first products
    for (int i = 0; i < 2; ++i) {
      Warp &w = warps[2 + i];
      Flight *mine = flight();
      int t = 0;
      bool here = false;
      auto arrive_x = [&] {
        if (!here) wait(w, cta[0].xf[t % XB], t / XB);
        here = true;
      };
      auto leave_x = [&] {
        arrive_x();
        commit(w, mine, cta[0].xe[t % XB], cta[1].xe[t % XB]);
        ++t;
        here = false;
      };
      for (int n = i, f = i; n < total; n += 2, f += 2) {
        for (; f >= blocks; f -= blocks) leave_x();
        const int p = n - NS;
        arrive_x();
        if (p >= 0) wait(w, cta[0].we[Order::slot(p)], Order::slot_phase(p));
        wait(w, cta[0].wf[Order::slot(n)], Order::slot_phase(n));
        commit(w, mine, cta[0].s[sums(n)], cta[1].s[sums(n)]);
      }
      while (t < tiles) leave_x();
    }
    // second products
    {
      Warp &w = warps[4];
      Flight *mine = flight();
      for (int n = 0; n < total; ++n) {
        const int f = n % blocks, t = n / blocks;
        if (f == 0 && t > 0) wait(w, cta[0].oe, t - 1);
        wait(w, cta[0].wf[Order::slot(n)], Order::slot_phase(n));
        wait(w, cta[0].h[Order::buffer(n)], Order::hidden_phase(n));
        commit(w, mine, cta[0].we[Order::slot(n)], cta[1].we[Order::slot(n)]);
        if (f == blocks - 1) commit(w, mine, cta[0].of, cta[1].of);
      }
    }
    // activations and results
    for (int k = 0; k < 4 * G; ++k) {
      Warp &w = warps[5 + k];
      const int r = k & 1, group = (k >> 1) & 1;
      int stored = 0;
      auto store_tile = [&](int t) {
        wait(w, cta[r].of, t);
        act(w, [this] { cta[0].oe.arrive(); });
      };
      int t = 0, f = group;
      for (int n = group; n < total; n += 2, f += 2) {
        while (f >= blocks) {
          f -= blocks;
          ++t;
        }
        for (; f > 0 && stored < t; ++stored) store_tile(stored);
        wait(w, cta[r].s[sums(n)], sums_phase(n));
        act(w, [this, n] { cta[0].h[Order::buffer(n)].arrive(); });
        for (; stored < t; ++stored) store_tile(stored);
      }
      for (; stored < tiles; ++stored) store_tile(stored);
    }
  }

  // false: it stood still
  bool run() {
    while (true) {
      double all = 0;
      std::vector<std::pair<double, std::function<void()>>> can;
      bool left = false;
      for (auto &w : warps) {
        if (w.steps.empty()) continue;
        left = true;
        if (!w.steps.front().ready()) continue;
        can.push_back({all += w.speed, [&w] {
                         auto s = w.steps.front();
                         w.steps.pop_front();
                         s.act();
                       }});
      }
      for (auto &f : flights)
        if (!f->work.empty())
          can.push_back({all += f->speed, [&f = *f] {
                           auto g = f.work.front();
                           f.work.pop_front();
                           g();
                         }});
      if (can.empty()) return !left;
      const double at = std::uniform_real_distribution<double>(0, all)(rng);
      size_t i = 0;
      while (i + 1 < can.size() && can[i].first < at) ++i;
      can[i].second();
      if (flights.size() > 64) {  // (copies that have landed)
        std::vector<std::unique_ptr<Flight>> keep;
        for (size_t j = 0; j < flights.size(); ++j)
          if (j < 3 || !flights[j]->work.empty()) keep.push_back(std::move(flights[j]));
        flights.swap(keep);
      }
    }
  }
  // Phases that did not end where the call ends.
  int wrong() {
    int n = 0;
    const int total = tiles * blocks;
    auto members = [&](int slots, int k) { return (total - k + slots - 1) / slots; };
    for (int k = 0; k < NS; ++k) n += cta[0].h[k].phase != members(NS, k);
    for (int r = 0; r < 2; ++r) n += cta[r].of.phase != tiles;
    return n + (cta[0].oe.phase != tiles);
  }
};

template <int NS, int NW, int XB, bool SHARED>
void all(unsigned seed, int runs) {
  int early = 0, still = 0, wrong = 0;
  for (int i = 0; i < runs; ++i) {
    std::mt19937 rng(seed + i);
    const int tiles = 1 + rng() % 5, blocks = 1 + rng() % 9;
    Model<NS, NW, XB, SHARED> m(tiles, blocks, rng());
    const bool done = m.run();
    early += m.early;
    still += !done;
    wrong += done && m.wrong();
  }
  std::printf("%d %d %d\n", early, still, wrong);
}

}  // namespace

int main(int, char **v) {
  const bool wide = std::atoi(v[1]) == 256, shared = std::atoi(v[2]) != 0;
  const unsigned seed = std::atoi(v[3]);
  const int runs = std::atoi(v[4]);
  if (wide)
    shared ? all<2, 3, 1, true>(seed, runs) : all<2, 3, 1, false>(seed, runs);
  else
    shared ? all<3, 5, 2, true>(seed, runs) : all<3, 5, 2, false>(seed, runs);
}
