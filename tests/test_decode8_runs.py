"""How decode8 cuts its work, on the host: decode8_runs.cuh compiled with g++ and run by a
scheduler that lets CTAs take their steps in any order.  Every tile is in one piece, a
unit's last piece merges it, and a launch in which CTAs give up leaves the arrival words
so that a replay of the same launch (a captured one has the same call id) is right."""

import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "grouped_query_attention_attn_b200", "csrc")

SOURCE = r"""
#include <cstdint>
#include <random>
#include <vector>
#include "decode8_runs.cuh"
using namespace gqa;

struct Word {
    unsigned long long *at;
    unsigned long long read() const { return *at; }
    void set(unsigned long long x) const { *at = x; }
    void cas(unsigned long long from, unsigned long long to) const { if (*at == from) *at = to; }
    unsigned long long add(unsigned long long x) const { const auto was = *at; *at += x; return was; }
};

struct Cta {
    D8Run run;
    D8Piece x;
    int b, step = 0, taken = 0;
    unsigned long long seen;
    bool done = false;
};

// One launch: units of n[b] tiles for Hkv heads, words[b * Hkv + h].  CTA c gives up in its
// give_up[c]-th piece (-1: never); leave: and arrives for none of what is left.  covered
// [B * Hkv * max_n] counts each tile's pieces, merged[unit] the merges, early the merges
// before every piece of this launch had arrived.  Returns early.
extern "C" int launch(const int *n, int B, int Hkv, int max_n, int ctas, int per, int total, const int *give_up,
                      int leave, unsigned long long id, unsigned long long *words, int *covered, int *merged,
                      unsigned seed) {
    std::mt19937 rng(seed);
    std::vector<int> arrived(B * Hkv, 0);
    std::vector<Cta> cta(ctas);
    auto tiles_of = [&](int b) { return n[b]; };
    auto word_of = [&](int b, int h) { return Word{words + b * Hkv + h}; };
    for (int c = 0; c < ctas; ++c) {
        D8Run &r = cta[c].run;
        r = {per * c, 0, 0, 0, 0};
        r.end = r.pos + per < total ? r.pos + per : total;
        int off = 0;
        if (r.pos < r.end)
            for (int b = 0; b < B; ++b) {
                const int each = n[b] ? n[b] + kD8Begin : 0;
                if (r.pos < off + each * Hkv) {
                    r.b = b;
                    r.kvh = (r.pos - off) / each;
                    r.tile0 = off + r.kvh * each + kD8Begin;
                    break;
                }
                off += each * Hkv;
            }
    }
    int early = 0, left = ctas;
    while (left) {
        const int c = rng() % ctas;
        Cta &t = cta[c];
        if (t.done) continue;
        const Word w = t.step ? word_of(t.b, t.x.head) : Word{nullptr};
        const int pieces = t.step ? t.x.cta1 - t.x.cta0 + 1 : 0;
        if (t.step == 0) {                          // the next piece
            for (t.x.count = 0; t.x.count <= 0;) {
                if (!(t.run.pos < t.run.end && t.run.b < B)) break;
                if (n[t.run.b] == 0) { ++t.run.b; continue; }
                t.b = t.run.b;
                t.x = d8_take(t.run, n[t.b], Hkv, per, c, ctas);
            }
            if (t.x.count <= 0) { t.done = true; --left; continue; }
            for (int i = 0; i < t.x.count; ++i) ++covered[(t.b * Hkv + t.x.head) * max_n + t.x.first + i];
            if (t.x.cta0 == t.x.cta1) {
                if (t.taken++ == give_up[c]) {
                    if (!leave) d8_abandon(t.run, B, Hkv, per, c, ctas, id, tiles_of, word_of);
                    t.done = true; --left;
                }
                continue;
            }
            t.step = 1;
        } else if (t.step == 1) {
            t.seen = w.read();
            t.step = 2;
        } else if (t.step == 2) {
            d8_claim(w, t.seen, id);
            t.step = 3;
        } else {
            const int unit = t.b * Hkv + t.x.head;
            t.step = 0;
            if (t.taken++ == give_up[c]) {
                if (!leave) {
                    d8_arrive(w, pieces, id);
                    d8_abandon(t.run, B, Hkv, per, c, ctas, id, tiles_of, word_of);
                }
                t.done = true; --left;
                continue;
            }
            ++arrived[unit];
            if (d8_arrive(w, pieces, id)) {
                ++merged[unit];
                early += arrived[unit] != pieces;
            }
        }
    }
    return early;
}
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    at = tmp_path_factory.mktemp("runs")
    (at / "runs.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-Wno-unused-parameter", "-fPIC", "-shared",
                    "-I", CSRC, str(at / "runs.cpp"), "-o", str(at / "runs.so")], check=True)
    lib = ctypes.CDLL(str(at / "runs.so"))
    lib.launch.argtypes = [ctypes.c_void_p] + [ctypes.c_int] * 6 + [ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64,
                                                                    ctypes.c_void_p, ctypes.c_void_p,
                                                                    ctypes.c_void_p, ctypes.c_uint]
    return lib


class Work:
    """A batch cut into runs as the kernel cuts it, and its arrival words."""

    def __init__(self, rng):
        self.B, self.Hkv, self.ctas = rng.randint(1, 7), rng.randint(1, 3), rng.choice([3, 8, 31])
        top = rng.choice([1, 5, 40, 300])
        self.n = [rng.choice([0, 1, top, rng.randint(1, top)]) for _ in range(self.B)]
        places = [x + 12 if x else 0 for x in self.n]
        self.total = sum(places) * self.Hkv
        least = int((0.25 * max(places)) ** 0.5)
        self.per = max((least + 4) // 4 * 4, (self.total - 1) // self.ctas + 1)
        self.max_n = max(max(self.n), 1)
        self.units = self.B * self.Hkv
        self.words = (ctypes.c_uint64 * self.units)(*(rng.getrandbits(64) for _ in range(self.units)))
        self.split = []                                # units in several pieces
        at = 0
        for b in range(self.B):
            for h in range(self.Hkv):
                at += 12 if self.n[b] else 0
                if self.n[b] and at // self.per != (at + self.n[b] - 1) // self.per:
                    self.split.append(b * self.Hkv + h)
                at += self.n[b]

    def launch(self, lib, rng, call_id, give_up=(), leave=False):
        up = (ctypes.c_int * self.ctas)(*([-1] * self.ctas))
        for c, i in give_up:
            up[c] = i
        covered = (ctypes.c_int * (self.units * self.max_n))()
        merged = (ctypes.c_int * self.units)()
        early = lib.launch((ctypes.c_int * self.B)(*self.n), self.B, self.Hkv, self.max_n, self.ctas, self.per,
                           self.total, up, int(leave), call_id, self.words, covered, merged, rng.getrandbits(32))
        return early, list(covered), list(merged)

    def right(self, result):
        early, covered, merged = result
        tiles = [int(i < self.n[u // self.Hkv]) for u in range(self.units) for i in range(self.max_n)]
        return early == 0 and covered == tiles and merged == [int(u in self.split) for u in range(self.units)]


def test_every_tile_once_and_one_merge(shim):
    rng = random.Random(1)
    for i in range(400):
        w = Work(rng)
        for _ in range(3):                             # replays of one launch
            assert w.right(w.launch(shim, rng, 77))
        assert w.right(w.launch(shim, rng, 78))


def gave_up(shim, leave):
    """How many replays after a launch in which CTAs gave up went wrong, of 400."""
    rng = random.Random(2)
    wrong = 0
    for i in range(400):
        w = Work(rng)
        w.launch(shim, rng, 77)
        who = [(c, rng.randint(0, 2)) for c in rng.sample(range(w.ctas), rng.randint(1, w.ctas))]
        w.launch(shim, rng, 77, give_up=who, leave=leave)
        if not leave:
            assert all(w.words[u] == 77 << 16 for u in w.split)
        wrong += not w.right(w.launch(shim, rng, 77))
    return wrong


def test_a_replay_after_ctas_gave_up_is_right(shim):
    assert gave_up(shim, leave=False) == 0


def test_a_cta_that_leaves_without_arriving_spoils_replays(shim):
    assert gave_up(shim, leave=True) > 100
