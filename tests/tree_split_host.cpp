// The split of tree attention over CTAs (csrc/tree_split.h), walked on the
// host: every item of every CTA's share.
#include "tree_split.h"

using namespace pa;

template <int G, int SEG_>
struct Shape {
    static constexpr int QPOS = kTreeRows / G, KT = kTreeKeys, SEG = SEG_;
};

// Items as rows of 10 ints: CTA, sequence, kv head, first draft, row tiles, j0,
// j1, key tiles, slot (-1: whole), pieces (0: no cut segment begins here).
template <class C>
static int walk_all(const TreeArgs &a, int ctas, int *out, int room) {
    int total = 0, n = 0;
    for (int b = 0; b < a.B; ++b) total += make_seq<C>(a, load_raw(a, b)).units_head(C::SEG) * a.Hkv;
    const int S = tree_share(total, ctas);
    for (int g = 0; g < ctas; ++g) {
        const int pos = (int)min((int64_t)g * S, (int64_t)total), end = min(total - pos, S) + pos;
        int b = 0, base = 0;
        for (int u; pos < end && pos >= base + (u = make_seq<C>(a, load_raw(a, b)).units_head(C::SEG) * a.Hkv); ++b) base += u;
        Walk<C> w{};
        Item it;
        w.start(a, pos, end, S, b, base);
        while (w.next(a, it)) {
            if (n == room) return -1;
            const int row[10] = {g, it.b, it.kvh, it.r0, it.rt, it.j0, it.j1, it.nt, it.whole() ? -1 : it.slot(g),
                                 it.begins_cut() ? w.pieces(it) : 0};
            for (int i = 0; i < 10; ++i) out[n * 10 + i] = row[i];
            ++n;
        }
    }
    return n;
}

extern "C" int tree_items(const int *cu_q, const int *prefix, int B, int max_blocks, int Hkv, int G, int max_q_len,
                          int total_q, int e4m3, int ctas, int *out, int room) {
    TreeArgs a{};
    a.cu_q = cu_q, a.prefix_lens = prefix, a.B = B, a.max_blocks = max_blocks, a.Hkv = Hkv, a.max_q_len = max_q_len;
    a.total_q = total_q;
    switch (G * 2 + e4m3) {
        case 2: return walk_all<Shape<1, kSegBf16>>(a, ctas, out, room);
        case 3: return walk_all<Shape<1, kSegE4m3>>(a, ctas, out, room);
        case 4: return walk_all<Shape<2, kSegBf16>>(a, ctas, out, room);
        case 5: return walk_all<Shape<2, kSegE4m3>>(a, ctas, out, room);
        case 8: return walk_all<Shape<4, kSegBf16>>(a, ctas, out, room);
        case 9: return walk_all<Shape<4, kSegE4m3>>(a, ctas, out, room);
        case 16: return walk_all<Shape<8, kSegBf16>>(a, ctas, out, room);
        case 17: return walk_all<Shape<8, kSegE4m3>>(a, ctas, out, room);
        default: return -2;
    }
}

extern "C" int tree_piece_slot_of(int cta, int p) { return tree_piece_slot(cta, p); }
