// A host model of a CTA of csrc/m2_attn_prompt_tile.cu: its warps run the ring's
// rules (m2_prompt_ring.h) and the tiles' meetings (m2_tile_meet.h) as threads over
// barriers that are waited on by parity, as the hardware's are, some of them slow.
// A wait that passes before its piece's turn is over is a fault, and so is a run
// that does not end. Prints "ok" and leaves 0 when there is none; `model pieces`
// gives refused pairs pieces of the ring, and `model full` lets the tiles wait for no
// more than their room to be empty, as checks that the model sees them.
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstring>
#include <functional>
#include <memory>
#include <mutex>
#include <thread>
#include <vector>

#include "m2_prompt_ring.h"
#include "m2_tile_meet.h"

using Clock = std::chrono::steady_clock;

// chunks of the tiles (tile 1: 0 when it has no rows); refused: rows, but no chunks
struct Pair {
    int chunks0, chunks1;
    bool refused;
    bool rows1;  // tile 1 has rows
    int chunks() const { return chunks1 > chunks0 ? chunks1 : chunks0; }
    int outputs() const { return rows1 ? 2 : 1; }
};

// One of the hardware's barriers of one arrival, waited on by parity.
struct Bar {
    int turns = 0;  // that are over
};

enum Slow { kNobody, kLanding, kLook, kLookRoom, kTile0, kTile1, kOperands };

struct Run {
    std::mutex mutex;
    std::condition_variable changed;
    Bar full[m2::kRingStages], empty[m2::kRingStages], ready[m2::kRingStages];
    int arrived[2] = {0, 0}, meeting[2] = {0, 0};  // three of a tile's warps complete a meeting
    int scores[2] = {0, 0}, outs[2] = {0, 0};      // chunks, and walks, whose products are done
    int known = 0, passed = 0;                     // pairs beyond the first that are known; warps that went on to them
    std::vector<int> landing;                      // pieces on their way
    bool over = false, early = false;
    int ended = 0;

    // everyone's waits end when the run is over
    bool wait(std::function<bool()> until) {
        std::unique_lock<std::mutex> lock(mutex);
        changed.wait(lock, [&] { return over || until(); });
        return !over;
    }
    void with(std::function<void()> f) {
        std::lock_guard<std::mutex> lock(mutex);
        f();
        changed.notify_all();
    }
    bool wait_turn(Bar& bar, int turn) {
        return wait([&] {
            if ((bar.turns & 1) == (turn & 1)) return false;
            if (bar.turns != turn + 1) early = true;
            return true;
        });
    }
};

// The ring as m2_prompt_ring.h sees it.
struct Ring {
    Run* run;
    static int at(int piece) { return piece % m2::kRingStages; }
    static int turn(int piece) { return piece / m2::kRingStages; }
    bool wait_full(int piece) { return run->wait_turn(run->full[at(piece)], turn(piece)); }
    bool wait_empty(int piece) { return run->wait_turn(run->empty[at(piece)], turn(piece)); }
    bool wait_ready(int piece) { return run->wait_turn(run->ready[at(piece)], turn(piece)); }
    void arrive_ready(int piece) {
        run->with([&] { ++run->ready[at(piece)].turns; });
    }
    void arrive_empty(int piece) {
        run->with([&] { ++run->empty[at(piece)].turns; });
    }
};

struct Meeting {
    Run* run;
    void sync(int i) const {
        std::unique_lock<std::mutex> lock(run->mutex);
        const int mine = run->meeting[i];
        if (++run->arrived[i] == 3) {
            run->arrived[i] = 0;
            ++run->meeting[i];
            run->changed.notify_all();
        } else {
            run->changed.wait(lock, [&] { return run->over || run->meeting[i] != mine; });
        }
    }
};

static void pause(bool yes) {
    if (yes) std::this_thread::sleep_for(std::chrono::milliseconds(2));
}

// 0: it ended; 1: a wait passed early; 2: it got stuck.
static int run_of(const std::vector<Pair>& pairs, Slow slow, bool refused_pieces, bool room_full) {
    std::shared_ptr<Run> run(new Run);
    const int count = (int)pairs.size();
    auto pieces_of = [=](const Pair& y) {
        if (refused_pieces && y.refused) return y.outputs();
        return m2::ring_pieces(y.chunks(), y.outputs());
    };
    // a warp's loop over the pairs
    auto every_pair = [=](std::function<void(const Pair&, int)> role) {
        for (int k = 0, first = 0; k < count; ++k) {
            role(pairs[k], first);
            first += pieces_of(pairs[k]);
            if (!run->wait([&] { return run->known > k; })) break;
            run->with([&] { ++run->passed; });
        }
        run->with([&] { ++run->ended; });
    };
    constexpr int kAhead = 3, kOthers = 5;
    std::vector<std::thread> warps;
    warps.emplace_back([=] {  // the copies
        Ring ring{run.get()};
        auto put = [&](const Pair& y, int first, int p) {
            run->with([&] {
                if (p >= 2 * y.chunks())
                    ++run->full[Ring::at(first + p)].turns;
                else
                    run->landing.push_back(first + p);
            });
        };
        for (int k = 0, first = 0; k < count; ++k) {
            const Pair& y = pairs[k];
            const int pieces = pieces_of(y), had = k > 0 ? std::min(kAhead, pieces) : 0, soon = std::min(m2::kRingStages, pieces);
            auto here = [&](int p) { put(y, first, p); };
            if (!m2::ring_fill(ring, first, had, soon, here)) break;
            if (k > 0 && !run->wait([&] { return run->passed >= kOthers * k; })) break;
            run->with([&] { run->known = k + 1; });
            if (!m2::ring_fill(ring, first, soon, pieces, here)) break;
            if (k + 1 < count) {
                const Pair& z = pairs[k + 1];
                if (!m2::ring_fill(ring, first + pieces, 0, std::min(kAhead, pieces_of(z)),
                                   [&](int p) { put(z, first + pieces, p); }))
                    break;
            }
            first += pieces;
        }
        run->with([&] { ++run->ended; });
    });
    warps.emplace_back([=] {  // the copies land
        for (;;) {
            if (!run->wait([&] { return !run->landing.empty(); })) return;
            pause(slow == kLanding);
            run->with([&] {
                ++run->full[Ring::at(run->landing.front())].turns;
                run->landing.erase(run->landing.begin());
            });
        }
    });
    warps.emplace_back([=] {  // what has landed, looked over
        every_pair([=](const Pair& y, int first) {
            Ring ring{run.get()};
            m2::ring_look(ring, first, pieces_of(y), [&](int p) { pause(slow == kLook || (slow == kLookRoom && p >= 2 * y.chunks() - 1)); });
        });
    });
    warps.emplace_back([=] {  // waits for the products' operands
        every_pair([=](const Pair& y, int first) {
            Ring ring{run.get()};
            m2::tile_turns_meet(Meeting{run.get()}, y.chunks(), y.chunks0, y.chunks1, [&](int j) {
                pause(slow == kOperands);
                if (j < y.chunks()) ring.wait_ready(first + 2 * j);
                if (j > 0) ring.wait_ready(first + 2 * j - 1);
            }, [](int, int) {});
        });
    });
    warps.emplace_back([=] {  // the products
        every_pair([=](const Pair& y, int first) {
            Ring ring{run.get()};
            m2::tile_turns_meet(Meeting{run.get()}, y.chunks(), y.chunks0, y.chunks1, [](int) {}, [&](int i, int j) {
                const int n = i ? y.chunks1 : y.chunks0;
                const bool last = i == 1 || y.chunks1 == 0;
                if (j > 0 && last) ring.arrive_empty(first + 2 * j - 1);
                if (j < n && last) ring.arrive_empty(first + 2 * j);
                run->with([&] { ++(j < n ? run->scores[i] : run->outs[i]); });
            });
        });
    });
    for (int i = 0; i < 2; ++i)
        warps.emplace_back([=] {  // a tile's softmax
            int chunks = 0, walks = 0, leaving = -1;
            Ring ring{run.get()};
            auto left = [&] {
                if (leaving >= 0) ring.arrive_empty(leaving);
                leaving = -1;
            };
            every_pair([&](const Pair& y, int first) {
                const int n = i ? y.chunks1 : y.chunks0;
                left();
                m2::tile_rows_meet(Meeting{run.get()}, i, n, [&](int j) { run->wait([&] { return run->scores[i] > chunks + j; }); });
                chunks += n;
                if (n > 0) {
                    const int mine = walks++;
                    run->wait([&] { return run->outs[i] > mine; });
                }
                if (i && !y.rows1) return;
                pause(slow == (i ? kTile1 : kTile0));
                if (pieces_of(y) == 0) return;
                const int piece = first + 2 * y.chunks() + i;
                if (room_full)
                    ring.wait_full(piece);
                else
                    m2::ring_room(ring, piece);
                leaving = piece;
            });
            left();
        });
    bool all;
    {
        std::unique_lock<std::mutex> lock(run->mutex);
        all = run->changed.wait_until(lock, Clock::now() + std::chrono::seconds(10), [&] { return run->early || run->ended == 6; });
        run->over = true;
        run->changed.notify_all();
    }
    for (std::thread& t : warps) t.join();
    return run->early ? 1 : all ? 0 : 2;
}

int main(int argc, char** argv) {
    const bool pieces = argc > 1 && !std::strcmp(argv[1], "pieces"), full = argc > 1 && !std::strcmp(argv[1], "full");
    const Pair refused = {0, 0, true, true}, refused1 = {0, 0, true, false};
    auto pair = [](int n0, int n1) { return Pair{n0, n1, false, n1 > 0}; };
    const std::vector<std::vector<Pair>> runs = {
        {pair(1, 1), pair(1, 1), pair(1, 1), pair(1, 1)},
        {pair(1, 0), pair(1, 0), pair(1, 0), pair(1, 0), pair(1, 0), pair(1, 1)},
        {pair(2, 3), pair(1, 0), pair(7, 7), pair(4, 0), pair(4, 5), pair(1, 1)},
        {pair(5, 0), refused, pair(5, 0), refused, pair(3, 3), pair(5, 0)},
        {pair(6, 0), refused1, refused, refused, pair(4, 4), refused, refused, refused, pair(1, 0), pair(2, 2)},
        {refused, refused, refused, pair(1, 1), pair(5, 0), refused, pair(1, 0)},
    };
    int faults = 0;
    for (size_t r = 0; r < runs.size(); ++r)
        for (int slow = kNobody; slow <= kOperands; ++slow) {
            const int what = run_of(runs[r], (Slow)slow, pieces, full);
            if (what == 0) continue;
            std::printf("%s: run %d, slow %d\n", what == 1 ? "early" : "stuck", (int)r, slow);
            ++faults;
            if (pieces || full) return 2;
        }
    if (!faults) std::printf("ok\n");
    return faults ? 1 : 0;
}
