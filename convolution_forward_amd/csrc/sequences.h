// Device-side view of packed sequences (internal.h, struct Sequences): where
// a sequence begins and ends, which state slot it uses, and how tiles that
// stay inside one sequence are numbered without knowing the lengths on the
// host.
#pragma once

#include "internal.h"

namespace convfwd {

// First row of sequence n (n <= num_seqs; n == num_seqs gives the end),
// clamped to the buffer whatever the offsets hold.
__device__ __forceinline__ int64_t seq_begin(const Sequences &s, int n)
{
    if (!s.offsets)
        return s.each * n;
    const int64_t v = s.offsets[n];
    return v < 0 ? 0 : (v > s.tokens ? s.tokens : v);
}

// The state slot of sequence n, or -1: none.
__device__ __forceinline__ int seq_slot(const Sequences &s, int n)
{
    const int v = s.slots ? s.slots[n] : n;
    return v >= 0 && v < s.num_slots ? v : -1;
}

// Tiles of at most `tile` rows of one sequence. Sequence n's tiles are
// numbered from begin(n) / tile + n on: since
//   floor((b + len) / tile) + 1 >= floor(b / tile) + ceil(len / tile),
// the next sequence's first number is past this one's last, every sequence
// (an empty one too) has at least one number, and tokens / tile + num_seqs
// numbers are enough. Numbers past a sequence's last tile name no rows.
struct SeqTile {
    int n;              // sequence
    int index;          // tile within the sequence; 0 also for an empty sequence
    int64_t begin, len; // the sequence's rows
};

inline int64_t seq_tiles(const Sequences &s, int tile) { return s.tokens / tile + s.num_seqs; }

// Sequences as a plan of sizes alone sees them: equally long, or with offsets,
// of which it only asks whether there are any.
inline Sequences sequences_of(int64_t tokens, int num_seqs, bool equal)
{
    static const int32_t some = 0;
    Sequences s = {};
    s.offsets = equal ? nullptr : &some;
    s.num_seqs = num_seqs;
    s.tokens = tokens;
    s.each = tokens / num_seqs;
    return s;
}

// Called by whole waves with a uniform number: 64 lanes probe 64 sequences at
// a time, so up to 64 sequences cost one memory round trip, 4096 two.
__device__ __forceinline__ SeqTile seq_tile(const Sequences &s, int tile, int number)
{
    // The last n with begin(n) / tile + n <= number (n = 0 always qualifies
    // for offsets that start at 0, and is where any others end up).
    const int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    int lo = 0, count = s.num_seqs;
    while (count > 64) {
        const int step = (count + 63) >> 6;
        const int at = lane * step;
        const bool ok = at < count && seq_begin(s, lo + (at < count ? at : 0)) / tile + lo + at <= number;
        const uint64_t yes = __ballot(ok);
        const int k = yes ? 63 - __builtin_clzll(yes) : 0;
        lo += k * step;
        count = min(step, count - k * step);
    }
    // The last 64: each lane looks at one sequence and at its end.
    const int mine = lo + (lane < count ? lane : 0);
    const int begin = (int)seq_begin(s, mine), end = (int)seq_begin(s, mine + 1);
    const uint64_t yes = __ballot(lane < count && begin / tile + mine <= number);
    const int k = yes ? 63 - __builtin_clzll(yes) : 0;
    SeqTile t;
    t.n = __builtin_amdgcn_readfirstlane(lo + k);
    t.begin = __builtin_amdgcn_readlane(begin, k);
    t.len = __builtin_amdgcn_readlane(end, k) - (int)t.begin;
    if (t.len < 0)
        t.len = 0;
    const int first = (int)(t.begin / tile) + t.n;
    t.index = number < first ? 0 : number - first;
    return t;
}

}  // namespace convfwd
