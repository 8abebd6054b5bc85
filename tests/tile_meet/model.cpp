// A host model of the tiles' meetings: the six warps of each of two tiles run
// csrc/m2_tile_meet.h as threads over a barrier that counts arrivals as the
// hardware's does, with bounded waits that run out wherever a run says so.
// Prints "ok" and leaves 0 when every warp of every run comes to its end;
// `model arrive` lets the softmax warps arrive without waiting, as a check that
// the model sees a protocol that gets stuck.
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstring>
#include <memory>
#include <mutex>
#include <thread>
#include <vector>

#include "m2_tile_meet.h"

using Clock = std::chrono::steady_clock;

// What one run shares; it outlives threads that are stuck.
struct Run {
    std::mutex mutex;
    std::condition_variable changed;
    int arrived[2] = {0, 0};  // warps counted for a tile's present meeting (6 complete it)
    int meeting[2] = {0, 0};
    int scores[2] = {0, 0};   // chunks whose products a tile's warps may read
    bool over = false;        // the run is given up
    int ended = 0;
};

struct Barrier {
    Run* run;
    bool wait = true;
    void sync(int i) const {
        std::unique_lock<std::mutex> lock(run->mutex);
        const int mine = run->meeting[i];
        if (++run->arrived[i] == 6) {
            run->arrived[i] = 0;
            ++run->meeting[i];
            run->changed.notify_all();
        } else if (wait) {
            run->changed.wait(lock, [&] { return run->meeting[i] != mine || run->over; });
        }
    }
};

static void pause_ms(int ms) {
    if (ms) std::this_thread::sleep_for(std::chrono::milliseconds(ms));
}

// chunks0, chunks1: of the tiles. fails: the chunk whose scores nobody waits
// for long enough (-1: none); slow: milliseconds that the operands of that
// chunk and of later ones take.
static bool run_ends(int chunks0, int chunks1, int fails, int slow, bool arrive) {
    std::shared_ptr<Run> run(new Run);
    const int chunks = chunks1 > 0 ? chunks1 : chunks0;
    std::vector<std::thread> warps;
    auto end = [run] {
        std::lock_guard<std::mutex> lock(run->mutex);
        ++run->ended;
        run->changed.notify_all();
    };
    for (int i = 0; i < 2; ++i)
        for (int w = 0; w < 4; ++w)
            warps.emplace_back([=] {
                bool good = true;
                m2::tile_rows_meet(Barrier{run.get(), !arrive}, i, i ? chunks1 : chunks0, [&](int j) {
                    if (j == fails) good = false;  // the wait has run out
                    if (!good) return;
                    std::unique_lock<std::mutex> lock(run->mutex);
                    run->changed.wait(lock, [&] { return run->scores[i] > j || run->over; });
                });
                end();
            });
    warps.emplace_back([=] {  // the products
        m2::tile_turns_meet(Barrier{run.get()}, chunks, chunks0, chunks1, [](int) {}, [&](int i, int j) {
            std::lock_guard<std::mutex> lock(run->mutex);
            run->scores[i] = j + 1;
            run->changed.notify_all();
        });
        end();
    });
    warps.emplace_back([=] {  // the operands
        m2::tile_turns_meet(Barrier{run.get()}, chunks, chunks0, chunks1,
                            [&](int j) { pause_ms(fails >= 0 && j >= fails ? slow : 0); }, [](int, int) {});
        end();
    });
    bool all;
    {
        std::unique_lock<std::mutex> lock(run->mutex);
        all = run->changed.wait_until(lock, Clock::now() + std::chrono::seconds(3), [&] { return run->ended == 10; });
        run->over = true;
        run->changed.notify_all();
    }
    for (std::thread& t : warps) t.join();
    return all;
}

int main(int argc, char** argv) {
    const bool arrive = argc > 1 && !std::strcmp(argv[1], "arrive");
    const int sizes[][2] = {{1, 1}, {4, 5}, {5, 5}, {0, 3}, {3, 0}, {2, 7}};
    int stuck = 0;
    for (const int* n : sizes)
        for (int fails = -1; fails < 7; ++fails)
            for (int slow = 0; slow < 12; slow += 10) {
                if (fails >= n[0] && fails >= n[1]) continue;
                if (run_ends(n[0], n[1], fails, slow, arrive)) continue;
                std::printf("stuck: %d and %d chunks, a wait runs out at chunk %d\n", n[0], n[1], fails);
                if (arrive) return 2;
                ++stuck;
            }
    if (!stuck) std::printf("ok\n");
    return stuck ? 1 : 0;
}
