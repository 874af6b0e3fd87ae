"""Host-only check of how parts of one result agree on the one that finishes it (part_words.h, and shared_word.h where
every part counts itself): the library's own headers, compiled for the host, with every part as a fiber that a random
scheduler stops before each access to shared memory. Some parts are not started until others have ended: the result
is finished exactly once all the same, by one that finds every part's sums written, and the words are zero
afterwards, for the next run under the same tag."""
import os
import subprocess

import w4a16_nvfp4_dense_amd as ffn

CSRC = os.path.join(ffn.PKG_DIR, "csrc")

MODEL = r"""
#include <ucontext.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <memory>
#include <random>
#include <vector>

#include "part_words.h"

using namespace ffn;

static int run_number;
#define CHECK(c) \
    do { \
        if (!(c)) { \
            std::printf("line %d: %s  (run %d)\n", __LINE__, #c, run_number); \
            std::exit(1); \
        } \
    } while (0)

static std::mt19937_64 rng(1);
static ucontext_t scheduler;
struct Fiber {
    ucontext_t at;
    std::unique_ptr<char[]> stack;
    int part;
    bool done;
};
static Fiber *running;
static void yield() { swapcontext(&running->at, &scheduler); }

typedef unsigned long long u64;
struct Word {
    u64 *at;
    u64 load() const { yield(); return *at; }
    void clear() const { yield(); *at = 0; }
    u64 swap(u64 v) const { yield(); const u64 old = *at; *at = v; return old; }
    u64 add_one() const { return add(1); }
    u64 add(int n) const { yield(); const u64 old = *at; *at += n; return old; }
    bool exchange(u64 &seen, u64 next) const
    {
        yield();
        if (*at == seen) {
            *at = next;
            return true;
        }
        seen = *at;
        return false;
    }
};

// One result: words 0 .. P - 2 of the lower parts, P - 1 of the last part.
static int P, looks;
static u64 tag;
static std::vector<u64> words;
static std::vector<int> sums;  // written (1) or not
static int finished;
static long in_registers;      // finishes of the last part without writing its sums

static void part(int i)
{
    const auto word = [](int k) { return Word{&words[k]}; };
    bool mine = false;
    if (i == P - 1) {
        mine = true;
        for (int k = 0; k < P - 1 && mine; ++k) {
            mine = false;
            for (int n = 0; n < looks && !mine; ++n)
                mine = word(k).load() == marked(tag);
        }
        if (mine)
            ++in_registers;
    }
    if (!mine) {
        yield();
        sums[i] = 1;
        if (i < P - 1) {
            const u64 was = word(i).swap(marked(tag));
            mine = was == given_up(tag) && late_part(word(P - 1), tag, P);
        } else {
            mine = last_gives_up(word, word(P - 1), tag, P);
        }
    }
    if (!mine)
        return;
    for (int k = 0; k < P; ++k) {
        yield();
        CHECK(sums[k] == 1 || (k == P - 1 && i == P - 1));
    }
    for (int k = 0; k < P; ++k)
        word(k).clear();
    ++finished;
}

// The other agreement (shared_word.h): every part writes and counts, in word 0.
static bool counting;
static void counted_part(int i)
{
    yield();
    sums[i] = 1;
    const Word word{&words[0]};
    if (count_part(word, tag, rng() % 2 ? 0 : words[0]) != P)
        return;
    for (int k = 0; k < P; ++k)
        CHECK(sums[k] == 1);
    word.clear();
    ++finished;
}

static void entry()
{
    Fiber *self = running;
    counting ? counted_part(self->part) : part(self->part);
    self->done = true;
    swapcontext(&self->at, &scheduler);
}

// All parts, at most `places` at a time, started in the order given.
static void run(const std::vector<int> &order, int places)
{
    std::vector<std::unique_ptr<Fiber>> live;
    size_t next = 0;
    finished = 0;
    sums.assign(P, 0);
    while (next < order.size() || !live.empty()) {
        while (static_cast<int>(live.size()) < places && next < order.size()) {
            auto f = std::make_unique<Fiber>();
            f->stack.reset(new char[32768]);
            getcontext(&f->at);
            f->at.uc_stack.ss_sp = f->stack.get();
            f->at.uc_stack.ss_size = 32768;
            f->at.uc_link = nullptr;
            f->part = order[next++];
            f->done = false;
            makecontext(&f->at, entry, 0);
            live.push_back(std::move(f));
        }
        const size_t i = rng() % live.size();
        running = live[i].get();
        for (int steps = rng() % 5; steps >= 0 && !running->done; --steps)
            swapcontext(&scheduler, &running->at);
        if (running->done) {
            live[i] = std::move(live.back());
            live.pop_back();
        }
    }
    CHECK(finished == 1);
    for (u64 w : words)
        CHECK(w == 0 || !is_tagged(w, tag));
}

int main()
{
    long gave_up = 0, runs = 0;
    for (run_number = 0; run_number < 20000; ++run_number) {
        rng.seed(run_number);
        P = 2 + rng() % 7;
        looks = rng() % 12;
        tag = tag_of_launch(rng());
        words.resize(P);
        for (u64 &w : words)  // zeros, anything, another launch's mark, giving up or count
            w = rng() % 3 == 0 ? 0 : rng() % 2 ? rng() : tag_of_launch(rng()) + (rng() % 2 ? 0xFFFF : rng() % 4);
        std::vector<int> order(P);
        for (int i = 0; i < P; ++i)
            order[i] = i;
        std::shuffle(order.begin(), order.end(), rng);
        const int places = 1 + rng() % P;
        in_registers = 0;
        counting = run_number % 4 == 3;
        for (int replay = 0; replay < 3; ++replay)  // the same tag on what the run before left
            run(order, places);
        for (u64 w : words)
            CHECK(!is_tagged(w, tag));
        if (!counting) {
            gave_up += 3 - in_registers;
            runs += 3;
        }
    }
    CHECK(gave_up > runs / 10 && gave_up < runs * 9 / 10);  // both ways are gone
    std::puts("ok");
    return 0;
}
"""


def test_finished_once(tmp_path):
    (tmp_path / "model.cpp").write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-O2", "-w", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", CSRC,
                    str(tmp_path / "model.cpp"), "-o", str(tmp_path / "model")], check=True)
    r = subprocess.run([str(tmp_path / "model")], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
