// The way out of a ring of copies (moe_ring.h) against a model of what it leaves:
// barriers with arrivals, bytes and phases, copies that land when they like, and
// threads that take turns in random order until one of them gives up.
//
//   ring_sim <mode> <seeds>     prints "ok", or the first seed that went wrong
//
// modes: "one" (a thread issues whole copies), "halves" (four threads, as the two
// kinds of moe_ring.h), and two mistakes that the model has to notice: "skipped"
// (copies that were never issued count as issued) and "early" (nobody is waited for).
#include "moe_ring.h"

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

namespace {

struct Barrier {
    int count = 1, pending = 1, bytes = 0, phase = 0;
    void settle()
    {
        if (pending == 0 && bytes == 0) {
            ++phase;
            pending = count;
        }
    }
    void arrive()
    {
        --pending;
        settle();
    }
    void expect(int n)
    {
        bytes += n;
        arrive();
    }
    void landed(int n)
    {
        bytes -= n;
        settle();
    }
    bool test(int parity) const { return (phase & 1) != parity; }
};

struct Copy {
    Barrier *bar;
    int bytes;
};

struct Sim {
    std::mt19937 rng;
    int stages;
    std::vector<Barrier> full, empty;
    std::vector<Copy> flying;
    bool abort = false;

    Sim(unsigned seed, int stages_, int halves) : rng(seed), stages(stages_), full(stages_), empty(stages_)
    {
        for (auto &b : full) b.count = b.pending = halves;
    }
    int pick(int n) { return static_cast<int>(rng() % static_cast<unsigned>(n)); }
    void land_one()
    {
        if (flying.empty()) return;
        const int i = pick(static_cast<int>(flying.size()));
        flying[i].bar->landed(flying[i].bytes);
        flying.erase(flying.begin() + i);
    }
    void issue(int n, int bytes)
    {
        Barrier &b = full[n % stages];
        if (pick(8) == 0) {  // a page out of range: an arrival, no copy
            b.arrive();
        } else {
            b.expect(bytes);
            flying.push_back({&b, bytes});
        }
    }
    // wait of the way out; false where it would run into its limit
    bool landed(int stage, int parity)
    {
        for (int i = 0; i < 1000; ++i) {
            if (full[stage].test(parity)) return true;
            land_one();
        }
        return false;
    }
};

// A producer takes the copies first, first + step, .. of `total`.
struct Producer {
    int next, step, issued = 0, past = 0;
    // one turn; false at the end
    bool turn(Sim &s, int total)
    {
        if (next >= total) return false;
        const int n = next;
        if (n >= s.stages && !s.abort && !s.empty[n % s.stages].test((n / s.stages - 1) & 1)) return true;
        if (!s.abort) {
            s.issue(n, 64);
            issued = n + 1;
        }
        past = n + 1;
        next += step;
        return true;
    }
};

bool run(const char *mode, unsigned seed)
{
    const bool halves = std::strcmp(mode, "halves") == 0, skipped = std::strcmp(mode, "skipped") == 0,
               early = std::strcmp(mode, "early") == 0;
    std::mt19937 r(seed * 7919u + 1u);
    const int stages = halves ? 4 * (1 + static_cast<int>(r() % 3u)) : 2 + static_cast<int>(r() % 9u);
    const int total = static_cast<int>(r() % 60u), give_up = static_cast<int>(r() % 200u);
    Sim s(seed, stages, halves ? 2 : 1);
    std::vector<Producer> p;
    if (halves)
        for (int i = 0; i < 4; ++i) p.push_back({i >> 1, 2});  // k and v of even copies, of odd ones
    else
        p.push_back({0, 1});
    int read = 0;  // copies that the readers are done with
    for (int t = 0;; ++t) {
        if (t == give_up) s.abort = true;
        bool more = false;
        const int who = s.pick(static_cast<int>(p.size()) + 2);
        if (who < static_cast<int>(p.size()))
            p[who].turn(s, total);
        else if (who == static_cast<int>(p.size()))
            s.land_one();
        else if (read < total && (s.abort || s.full[read % stages].test((read / stages) & 1)))
            s.empty[read++ % stages].arrive();
        for (auto &q : p) more |= q.next < total;
        // all threads have met (the readers too, where nobody gave up)
        if (!more && (s.abort || read == total)) break;
    }
    bool ok = true;
    if (s.abort && !early) {
        auto wait = [&](int st, int parity) { ok = s.landed(st, parity) && ok; };
        if (halves)
            for (int odd = 0; odd < 2; ++odd)
                moe::ring_drain_halves(odd, p[2 * odd].issued, p[2 * odd + 1].issued, stages,
                                       [&](int st) { s.full[st].arrive(); }, wait);
        else
            moe::ring_drain(skipped ? p[0].past : p[0].issued, stages, wait);
    }
    return ok && s.flying.empty();
}

}  // namespace

int main(int argc, char **argv)
{
    const char *mode = argc > 1 ? argv[1] : "one";
    const int seeds = argc > 2 ? std::atoi(argv[2]) : 1000;
    for (int i = 0; i < seeds; ++i)
        if (!run(mode, static_cast<unsigned>(i))) {
            std::printf("seed %d\n", i);
            return 0;
        }
    std::printf("ok\n");
    return 0;
}
