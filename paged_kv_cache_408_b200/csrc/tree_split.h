// tree_split.h -- how tree attention (tree.cu) cuts a batch into the CTAs'
// shares.  Integers only; compiled for the device and, for the tests, for the
// host.
//
// The segments (sequence, kv head, one or two row tiles of 128 rows) form one
// line of cost units: SEG at a segment's head, then kOne or kPair a key tile.
// The line is cut into equal contiguous shares; a tile belongs to the share
// that holds its first unit.
#pragma once

#include "pa.h"
#include "kernels.h"

#ifdef __CUDACC__
#define PA_SPLIT __host__ __device__ __forceinline__
#else
#include <algorithm>
#define PA_SPLIT inline
using std::max;
using std::min;
#endif

namespace pa {
namespace {

constexpr int kTreeRows = 128, kTreeKeys = 128;  // of a row tile, of a key tile
// line units of a key tile, in a segment of one and of two row tiles
constexpr int kOne = 2, kPair = 3;
// line units of a segment itself, by cache type (measured: tree.cu)
constexpr int kSegBf16 = 5, kSegE4m3 = 7;

// Units of a CTA's share: at least a tile's.
PA_SPLIT int tree_share(int total, int ctas) { return max((total + ctas - 1) / ctas, kPair); }

// Slot of CTA `cta`'s partial result of a cut segment: of the segments a CTA
// meets only its last can go on behind its share (the segment's first piece),
// only its first can have begun before it (a later one).
PA_SPLIT int tree_slot(int cta, bool first_piece) { return cta * 2 + (first_piece ? 1 : 0); }
// That of piece p of the cut segment that begins in CTA `cta`.
PA_SPLIT int tree_piece_slot(int cta, int p) { return tree_slot(cta + p, p == 0); }

// A sequence of the batch: its metadata as loaded, and checked.
struct Raw {
    int q0, q1, P;
};
struct Seq {
    int q0, T, P;          // first row, drafts (0 if its metadata is bad), prefix
    bool bad;
    int nt, npair, none;   // key tiles; segments of two and of one row tile per kv head
    PA_SPLIT int units_head(int seg) const { return npair * (seg + nt * kPair) + none * (seg + nt * kOne); }
};

PA_SPLIT Raw load_raw(const TreeArgs &a, int b) {
    b = min(b, a.B - 1);
    return {a.cu_q[b], a.cu_q[b + 1], a.prefix_lens[b]};
}

template <class C>
PA_SPLIT Seq make_seq(const TreeArgs &a, const Raw &x) {
    Seq s;
    const int64_t T = (int64_t)x.q1 - x.q0;
    s.bad = x.q0 < 0 || T < 0 || T > a.max_q_len || x.q1 > a.total_q || x.P < 0 ||
            x.P + T > (int64_t)a.max_blocks * 16;
    s.q0 = x.q0;
    s.T = s.bad ? 0 : (int)T;
    s.P = s.bad ? 0 : x.P;
    const int nmt = (s.T + C::QPOS - 1) / C::QPOS;
    s.npair = nmt >> 1;
    s.none = nmt & 1;
    s.nt = (s.P + s.T + C::KT - 1) / C::KT;
    return s;
}

// Key tiles [j0, j1) of one segment.
struct Item {
    int b, kvh, q0, T, P, L;   // q0: first row of the segment; T: drafts of the sequence
    int r0, rt;                // first draft of the segment; its row tiles, 1 or 2
    int j0, j1, nt;            // nt: key tiles of the segment
    int tile0;                 // line position of its first tile
    PA_SPLIT int steps() const { return (j1 - j0) * rt; }
    PA_SPLIT bool whole() const { return j0 == 0 && j1 == nt; }
    PA_SPLIT bool begins_cut() const { return j0 == 0 && j1 != nt; }
    PA_SPLIT int slot(int cta) const { return tree_slot(cta, j0 == 0); }
};

// Walks a CTA's share of the line.
template <class C>
struct Walk {
    int pos, end, base;  // base: line position of sequence b
    int S, b;
    Seq s;
    Raw nxt;                 // sequence b + 1, loaded ahead

    PA_SPLIT void start(const TreeArgs &a, int pos_, int end_, int S_, int b0, int base0) {
        pos = pos_, end = end_, S = S_, b = b0, base = base0;
        if (pos < end) {
            s = make_seq<C>(a, load_raw(a, b));
            nxt = load_raw(a, b + 1);
        }
    }
    PA_SPLIT bool next(const TreeArgs &a, Item &it) {
#pragma unroll 1
        while (pos < end) {
            const int head = s.units_head(C::SEG), off = pos - base;
            if (off >= head * a.Hkv) {
                base += head * a.Hkv;
                s = make_seq<C>(a, nxt);
                nxt = load_raw(a, ++b + 1);
                continue;
            }
            it.kvh = off / head;
            int r = off - it.kvh * head;           // unit within the kv head's segments, then within the segment
            const int Up = C::SEG + s.nt * kPair;
            int seg = r / Up;
            it.rt = seg < s.npair ? 2 : 1;
            seg = min(seg, s.npair);
            r -= seg * Up;
            const int wt = it.rt == 2 ? kPair : kOne, U = C::SEG + s.nt * wt;
            const int stop = min(U, end - pos + r);
            // the tiles whose first unit lies in the share
            it.j0 = max(0, r - C::SEG + wt - 1) / wt;
            it.j1 = max(0, stop - C::SEG + wt - 1) / wt;
            const int seg0 = pos - r;
            pos = seg0 + stop;
            if (it.j1 <= it.j0) continue;
            it.b = b;
            it.r0 = 2 * seg * C::QPOS;
            it.q0 = s.q0 + it.r0;
            it.T = s.T;
            it.P = s.P;
            it.L = s.P + s.T;
            it.nt = s.nt;
            it.tile0 = seg0 + C::SEG;
            return true;
        }
        return false;
    }
    // pieces of a segment: one for every share from the one that holds its
    // first tile's first unit to the one that holds its last tile's
    PA_SPLIT int pieces(const Item &it) const {
        const int last = it.tile0 + (it.nt - 1) * (it.rt == 2 ? kPair : kOne);
        return last / S - it.tile0 / S + 1;
    }
};

}  // namespace
}  // namespace pa
