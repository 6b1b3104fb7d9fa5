// decode8_runs.cuh -- how decode8 cuts its work: the tiles that a sequence reads, the
// pieces of units in a CTA's run, and the count of a unit's pieces.  Plain integer
// code, compiled for the host too.
#pragma once

#ifndef __CUDACC__
#define __host__
#define __device__
#define __forceinline__ inline
#endif

namespace gqa {

constexpr int kD8Keys = 32;                        // keys per tile
// What beginning a unit costs, in tiles.  8 and 16 were better and worse by up to 10 % on
// short sequences, by their lengths, and equal on long ones.
constexpr int kD8Begin = 12;

// Tiles a sequence of L keys reads, in order: those of the sinks
// below the window, then those from the window's first key on.
struct D8Tiles {
    int lo, sinks;              // key j is visible iff j < L and (j >= lo or j < sinks)
    int n_sink, first, n;       // sink tiles, first window tile, tiles in all
    __host__ __device__ D8Tiles(int L, int window, int n_sinks) {
        lo = window > 0 && L > window ? L - window : 0;
        sinks = window > 0 ? n_sinks : 0;
        const int below = sinks < lo ? sinks : lo;
        n_sink = (below + kD8Keys - 1) / kD8Keys;
        first = lo / kD8Keys > n_sink ? lo / kD8Keys : n_sink;
        const int last = L / kD8Keys + (L % kD8Keys > 0);
        n = n_sink + (last > first ? last - first : 0);
    }
    __host__ __device__ int tile(int i) const { return i < n_sink ? i : first + (i - n_sink); }
};

// A CTA's run, places pos .. end - 1 of the line of all units' places (kD8Begin empty ones
// and its tiles for each), and the unit that pos lies in or before: K/V head kvh of
// sequence b, first tile at place tile0.
struct D8Run {
    int pos, end, b, kvh, tile0;
};

// Tiles first .. first + count - 1 of K/V head `head` of the sequence; the unit is held by
// the runs of CTAs cta0 .. cta1.  count <= 0: empty places only.
struct D8Piece {
    int head, first, count, cta0, cta1;
};

// The run's next piece, in sequence run.b of n > 0 tiles; moves the run on, to the next
// sequence too.  per: places of each run; ctas: runs.
__host__ __device__ __forceinline__ D8Piece d8_take(D8Run &run, int n, int Hkv, int per, int cta, int ctas) {
    D8Piece x;
    const int unit_end = run.tile0 + n, stop = unit_end < run.end ? unit_end : run.end;
    x.head = run.kvh;
    x.first = run.pos > run.tile0 ? run.pos - run.tile0 : 0;
    x.count = stop - (run.tile0 + x.first);
    x.cta0 = x.cta1 = cta;
    if (x.first > 0) x.cta0 = run.tile0 / per;
    if (unit_end > run.end) {
        x.cta1 = (unit_end - 1) / per;
        if (x.cta1 > ctas - 1) x.cta1 = ctas - 1;
    }
    run.pos = stop;                                 // (a run may end in the empty places)
    if (stop == unit_end) {                         // on to the next unit
        run.tile0 = unit_end + kD8Begin;
        if (++run.kvh == Hkv) {
            run.kvh = 0;
            ++run.b;
        }
    }
    return x;
}

// Arrival word of a unit in several pieces: call id in the high 48 bits, arrivals in the
// low 16.  Every piece claims the word for this call before it starts (whatever
// another call, or uninitialised memory, left there; if the exchange fails, another
// piece has claimed it), so that an arrival is one addition.  The last one leaves
// (call id, 0) for a replay of the same launch, whose id is the same: so every piece
// has to arrive, whatever becomes of its CTA.  Word: read(), cas(from, to), add(x)
// (returns what was there) and set(x).
template <class Word>
__host__ __device__ __forceinline__ void d8_claim(Word word, unsigned long long seen, unsigned long long call_id) {
    if ((seen >> 16) != call_id) word.cas(seen, call_id << 16);
}

// True for the last of the unit's pieces.
template <class Word>
__host__ __device__ __forceinline__ bool d8_arrive(Word word, int pieces, unsigned long long call_id) {
    const bool last = static_cast<int>(word.add(1ull) & 0xFFFFu) + 1 == pieces;
    if (last) word.set(call_id << 16);
    return last;
}

// Arrives for every piece left of a run whose CTA gives up; what the pieces would have
// written is missing.  tiles_of(b): tiles of sequence b; word_of(b, head): a unit's word.
template <class TilesOf, class WordOf>
__host__ __device__ void d8_abandon(D8Run run, int B, int Hkv, int per, int cta, int ctas,
                                    unsigned long long call_id, TilesOf tiles_of, WordOf word_of) {
    while (run.pos < run.end && run.b < B) {
        const int b = run.b, n = tiles_of(b);
        if (n == 0) {
            ++run.b;
            continue;
        }
        const D8Piece x = d8_take(run, n, Hkv, per, cta, ctas);
        if (x.count <= 0 || x.cta0 == x.cta1) continue;
        const auto word = word_of(b, x.head);
        d8_claim(word, word.read(), call_id);
        d8_arrive(word, x.cta1 - x.cta0 + 1, call_id);
    }
}

}  // namespace gqa
