"""Host-only checks of how the int8 product's tiles are split and of how workgroups that share a tile agree on the
one that finishes it: the library's own header (int8_split.h), compiled for the host, with every workgroup of
several launches as a fiber that a random scheduler stops before each access to shared memory.

The model of the card: 8 XCDs, workgroup b of a launch on XCD b % 8, those of a launch started in order on each
XCD, a fixed number at a time over all launches, and a started one keeps its place until it ends. Nothing may
depend on which launch is started first on which XCD."""
import os
import subprocess

import pytest

import w4a16_nvfp4_dense_amd as ffn

CSRC = os.path.join(ffn.PKG_DIR, "csrc")

MODEL = r"""
#include <ucontext.h>

#include <cstdio>
#include <cstdlib>
#include <memory>
#include <random>
#include <vector>

#include "int8_split.h"

using namespace ffn;

#define CHECK(c) \
    do { \
        if (!(c)) { \
            std::printf("line %d: %s  (%s)\n", __LINE__, #c, label); \
            std::exit(1); \
        } \
    } while (0)

static char label[200];
static std::mt19937_64 rng(1);

struct Part {
    int b, tile, k, k_end;
};

// Every workgroup's parts in the order of its walk.
static std::vector<std::vector<Part>> walks(const Plan &p)
{
    std::vector<std::vector<Part>> all(p.groups);
    const Split &s = p.split;
    for (int b = 0; b < p.groups; ++b) {
        if (s.whole * s.stages + share(s, b + 1) - share(s, b) == 0)
            continue;
        Cursor at;
        at.start(s, b, p.groups);
        do
            all[b].push_back({b, at.tile, at.k, at.k_end});
        while (at.advance(s, b, p.groups, at.k_end - at.k));
    }
    return all;
}

// Units once each, the parts of a tile where the header says they are, slots
// that no two parts have, and how many parts a tile has at most.
static void check_split(const Plan &p)
{
    const Split &s = p.split;
    const long tiles = static_cast<long>(s.tiles_m) * s.tiles_n;
    const auto all = walks(p);
    std::vector<std::vector<Part>> of(tiles);
    for (const auto &w : all)
        for (const Part &x : w) {
            CHECK(x.tile >= 0 && x.tile < tiles && x.k >= 0 && x.k < x.k_end && x.k_end <= s.stages);
            of[x.tile].push_back(x);  // (by rising workgroup)
        }
    std::vector<int> slots(2 * s.sharers, 0);
    size_t most = 0;
    for (long t = 0; t < tiles; ++t) {
        int k = 0;
        for (const Part &x : of[t]) {
            CHECK(x.k == k);
            k = x.k_end;
        }
        CHECK(k == s.stages);
        most = std::max(most, of[t].size());
        if (of[t].size() == 1)
            continue;
        const int n = static_cast<int>(t) - s.whole * p.groups;
        CHECK(n >= 0 && n < s.shared);
        const Sharers in = sharers_of(s, n);
        CHECK(in.first == of[t].front().b && in.last == of[t].back().b);
        CHECK(static_cast<size_t>(in.last - in.first + 1) == of[t].size());
        CHECK(of[t].size() < (1u << kCountBits) - 1);
        for (size_t i = 0; i < of[t].size(); ++i) {
            const int b = of[t][i].b, slot = slot_number(s, in, b);
            CHECK(slot >= 0 && slot < 2 * s.sharers && !slots[slot]++);
            for (size_t j = 0; j + 1 < of[t].size(); ++j)
                CHECK(other_sharer(in, b, static_cast<int>(j)) == of[t][j < i ? j : j + 1].b);
        }
    }
    if (s.whole > 0)
        CHECK(most <= 3);
    else if (tiles >= p.groups)
        CHECK(most <= 2);
}

// ------------------------------------------------------------------ launches
struct Fiber {
    ucontext_t at;
    std::unique_ptr<char[]> stack;
    bool done = false;
};
static ucontext_t scheduler;
static Fiber *running;

static void yield() { swapcontext(&running->at, &scheduler); }

struct Word {
    unsigned long long *at;
    bool exchange(unsigned long long &seen, unsigned long long next) const
    {
        yield();
        if (*at == seen) {
            *at = next;
            return true;
        }
        seen = *at;
        return false;
    }
    unsigned long long add(int n) const
    {
        yield();
        const unsigned long long old = *at;
        *at += n;
        return old;
    }
    unsigned long long swap(unsigned long long v) const
    {
        yield();
        const unsigned long long old = *at;
        *at = v;
        return old;
    }
    unsigned long long load() const
    {
        yield();
        return *at;
    }
};

static long in_registers, written;  // tiles whose last workgroup found all others, and those where it gave up

struct Launch {
    Plan p;
    std::vector<std::vector<Part>> all;
    std::vector<unsigned long long> words;
    std::vector<long> slots;     // sums of k from k to k_end, or garbage
    std::vector<int> finished;   // of every tile
    int next[kXcds];             // workgroup to start on each XCD
};

static long sums(int k, int k_end)
{
    long v = 0;
    for (; k < k_end; ++k)
        v += 1000 + k;
    return v;
}

// What a workgroup does, without the products.
static void workgroup(Launch &l, int b)
{
    const Split &s = l.p.split;
    for (const Part &x : l.all[b]) {
        yield();
        long sum = sums(x.k, x.k_end);
        if (x.k > 0 || x.k_end < s.stages) {
            const int t = x.tile - s.whole * l.p.groups;
            const Sharers in = sharers_of(s, t);
            const int parts = in.last - in.first + 1;
            CHECK(parts <= 256);  // (as many threads as the smallest workgroup clear the words)
            const auto word = [&](int i) { return Word{&l.words[slot_number(s, in, in.first + i)]}; };
            bool mine = b == in.last;
            for (int i = 0; i + 1 < parts && mine; ++i) {
                mine = false;
                for (int looks = rng() % 40; looks > 0 && !mine; --looks)
                    mine = word(i).load() == marked(s.tag);
            }
            if (b == in.last)
                ++(mine ? in_registers : written);
            if (!mine) {
                yield();
                l.slots[slot_number(s, in, b)] = sum;
                mine = b == in.last ? last_gives_up(word, word(parts - 1), s.tag, parts)
                                    : word(b - in.first).swap(marked(s.tag)) == given_up(s.tag) &&
                                          late_part(word(parts - 1), s.tag, parts);
            }
            if (!mine)
                continue;
            for (int i = 0; i < parts; ++i) {
                yield();
                *word(i).at = 0;
            }
            for (int i = 0; i + 1 < parts; ++i) {
                yield();
                sum += l.slots[slot_number(s, in, other_sharer(in, b, i))];
            }
        }
        CHECK(sum == sums(0, s.stages));
        ++l.finished[x.tile];
    }
}

static Launch *entry_launch;
static int entry_b;
static void entry()
{
    Launch &l = *entry_launch;
    const int b = entry_b;
    Fiber *self = running;
    workgroup(l, b);
    self->done = true;
    swapcontext(&self->at, &scheduler);
}

// Runs the launches beside each other, `places` workgroups of an XCD at a time.
static void run(std::vector<Launch> &launches, int places)
{
    struct Running {
        std::unique_ptr<Fiber> f;
        int xcd;
    };
    std::vector<Running> live;
    int used[kXcds] = {};
    for (Launch &l : launches) {
        std::fill(l.finished.begin(), l.finished.end(), 0);
        std::fill(l.slots.begin(), l.slots.end(), -1);  // what an earlier launch left is wrong
        for (int x = 0; x < kXcds; ++x)
            l.next[x] = x;
    }
    for (;;) {
        // start whatever there is a place for, from a launch taken at random;
        // a launch that is favoured on an XCD may fill it alone
        for (int x = 0; x < kXcds; ++x)
            while (used[x] < places) {
                std::vector<Launch *> ready;
                for (Launch &l : launches)
                    if (l.next[x] < l.p.groups)
                        ready.push_back(&l);
                if (ready.empty())
                    break;
                Launch *l = rng() % 4 ? ready[x * 7 % ready.size()] : ready[rng() % ready.size()];
                Running r{std::make_unique<Fiber>(), x};
                r.f->stack.reset(new char[32768]);
                getcontext(&r.f->at);
                r.f->at.uc_stack.ss_sp = r.f->stack.get();
                r.f->at.uc_stack.ss_size = 32768;
                r.f->at.uc_link = nullptr;
                makecontext(&r.f->at, entry, 0);
                entry_launch = l;
                entry_b = l->next[x];
                l->next[x] += kXcds;
                ++used[x];
                running = r.f.get();
                swapcontext(&scheduler, &running->at);  // up to its first access
                live.push_back(std::move(r));
            }
        if (live.empty())
            break;
        const size_t i = rng() % live.size();
        running = live[i].f.get();
        for (int steps = rng() % 6; steps >= 0 && !running->done; --steps)
            swapcontext(&scheduler, &running->at);
        if (running->done) {
            --used[live[i].xcd];
            live[i] = std::move(live.back());
            live.pop_back();
        }
    }
    for (Launch &l : launches) {
        for (int n : l.finished)
            CHECK(n == 1);
        for (unsigned long long w : l.words)
            CHECK(!is_tagged(w, l.p.split.tag));
    }
}

int main()
{
    // every split of these ranges
    const int sizes[][4] = {{16, 128, 128, 256}, {16, 64, 64, 256}, {32, 128, 64, 256}, {64, 64, 64, 256},
                            {128, 128, 64, 256}, {128, 64, 64, 256}, {256, 128, 128, 256}, {256, 256, 256, 256},
                            {256, 256, 128, 304}, {16, 64, 64, 8}, {128, 128, 128, 7}, {64, 128, 128, 1}};
    for (const auto &z : sizes)
        for (int M : {1, 17, 64, 300, 2048, 4099})
            for (int K : {16, 128, 144, 640, 4112, 5120, 17408, 65536})
                for (int N : {1, 16, 333, 4099, 5120, 17408, 21504}) {
                    if (M > 20 * z[0])
                        continue;
                    std::snprintf(label, sizeof label, "M %d K %d N %d tile %d x %d cus %d", M, K, N, z[0], z[1], z[3]);
                    check_split(int8_plan(M, K, N, z[0], z[1], z[2], z[3]));
                }
    // divisions
    for (uint32_t d : {1u, 2u, 3u, 7u, 33u, 40u, 136u, 512u, 8 * 16384u})
        for (uint32_t n : {0u, 1u, d - 1, d, d + 1, 7 * d - 1, 7 * d, 0x7FFFFFFFu})
            CHECK(divisor(d).divide(n) == n / d);
    CHECK(tag_of_launch(0) != 0 && tag_of_launch(0xFFFF) != 0);
    // launches beside each other, and again and again on the same words
    const int shapes[][4] = {{1, 4096, 256, 1}, {1, 1664, 1000, 1}, {40, 2176, 900, 2}, {300, 4224, 1100, 3}};
    for (int seed = 0; seed < 60; ++seed) {
        rng.seed(seed);
        const auto &z = shapes[seed % 4];
        const int places = 1 + seed % 3;
        std::vector<Launch> launches(1 + seed % 5);
        std::snprintf(label, sizeof label, "run %d", seed);
        int n = 0;
        for (Launch &l : launches) {
            l.p = int8_plan(z[0], z[1] + 128 * n, z[2], 64, 64, 64, kXcds * places);
            l.p.split.tag = tag_of_launch(rng());
            l.all = walks(l.p);
            l.words.resize(2 * l.p.split.sharers);
            for (auto &w : l.words)  // zeros, anything, another launch's mark, giving up or count
                w = rng() % 3 == 0 ? 0 : rng() % 2 ? rng() : tag_of_launch(rng()) + (rng() % 2 ? 0xFFFF : rng() % 4);
            l.slots.resize(2 * l.p.split.sharers);
            l.finished.resize(l.p.split.tiles_m * l.p.split.tiles_n);
            ++n;
        }
        for (int replay = 0; replay < 3; ++replay) {  // the same tags on the words that the run before left
            run(launches, places);
            for (Launch &l : launches)
                for (int t = 0; t < l.p.split.shared; ++t) {
                    const Sharers in = sharers_of(l.p.split, t);
                    for (int w = in.first; w <= in.last && in.first != in.last; ++w)
                        CHECK(!is_tagged(l.words[slot_number(l.p.split, in, w)], l.p.split.tag));
                }
        }
    }
    CHECK(in_registers > 100 && written > 100);
    std::puts("ok");
    return 0;
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    at = tmp_path_factory.mktemp("int8_split")
    (at / "model.cpp").write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-O2", "-w", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", CSRC,
                    str(at / "model.cpp"), "-o", str(at / "model")], check=True)
    return str(at / "model")


def test_split_and_finishing(model):
    r = subprocess.run([model], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
