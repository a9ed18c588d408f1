// tree.cu -- attention of drafted tokens over a paged prefix and over the
// drafts each one may see (verification of a token tree), on the sm_100a
// tensor cores.
//
// Row i of sequence b (rows cu_q[b] .. cu_q[b+1]-1, T_b of them, at most 64)
// attends, per query head, to keys [0, P_b) and to key P_b + j for every
// draft j with bit j of mask[row] set:
//     out = sum_t softmax_t(scale q . k_t) v_t    over those keys,
// zero where there are none.
//
// Work split: a segment is (sequence, kv head, row tile), a row tile being
// 128 accumulator rows = 128/G drafts x the G query heads of a kv head, so
// K and V are read from HBM once per sequence (a second row tile, T G > 128,
// finds them in L2).  The segments' key tiles (128 keys, 8 blocks) form one
// line, kSegCost units at the head of each segment and one per tile, cut
// into equal contiguous shares, one per SM.  Of the segments a CTA meets
// only its first can have begun before its share and only its last can go
// on behind it, so two slots a CTA hold every partial result, whatever the
// batch; the merge kernel joins them by log-sum-exp.
//
// Within a CTA: a loader warp gathers K and V tiles through the block table
// (2-D TMA boxes, 128-byte swizzle) into two rings; one thread issues the
// MMAs; two softmax warpgroups take the key tiles in turn, each with its own
// score buffer, running maximum, sum and output accumulator in TMEM (a
// thread owns a whole row of 128 scores: no exchange between threads until
// the end of the segment, where the two accumulators are joined).  Scores of
// tile n+1 are computed while the exponentials of tile n run.  P is written
// over its scores in TMEM and is the A operand of P.V.  Warps whose 32 rows
// are all past the drafts skip the arithmetic.
// An E4M3 cache: the codes land in a staging ring and four warps widen them
// exactly to f16 operand tiles; the query rows are scaled by a power of two
// into f16's range.
// Bound: HBM for up to 128 rows a kv head (the tensor pipe then needs about
// a third of the time that the K and V bytes take), the tensor and softmax
// pipes beyond.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units the running maximum may lag behind
constexpr int kSegCost = 1;                // units charged per segment (query tile, epilogue)
constexpr int kMaxCtas = 160;              // partial-result slots: two a CTA
constexpr int kEpiBar = 1;                 // named barrier of the softmax warps
constexpr unsigned kFull = 0xffffffffu;

template <int D_, int G_, bool FP8_>
struct TCfg {
    static constexpr int D = D_, G = G_;
    static constexpr bool FP8 = FP8_;
    static constexpr int M = 128, KT = 128, BPT = KT / 16;
    static constexpr int QPOS = M / G;             // drafts of a row tile
    static constexpr int NATOM = D / 64;           // 128-byte column atoms along D
    static constexpr int ATOM = 128 * 128;         // bytes of one atom column of a 128-row tile
    static constexpr int TILE = NATOM * ATOM;      // a Q, K or V operand tile
    static constexpr int CODES = KT * D;           // a tile of E4M3 codes
    // rings: together about 192 KB, so that the copies in flight cover the
    // HBM latency (an SM's share of the bandwidth is ~24 B a clock)
    static constexpr int NSK = FP8 ? 2 : (D == 128 ? 3 : 6), NSV = NSK;
    static constexpr int NST = FP8 ? (D == 128 ? 4 : 12) : 0;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = TILE;
    static constexpr int OFF_V = OFF_K + NSK * TILE;
    static constexpr int OFF_C = OFF_V + NSV * TILE;
    static constexpr int OFF_ML = OFF_C + NST * CODES;     // [2][128] (m, l) of the two softmax warpgroups
    static constexpr int OFF_QEXP = OFF_ML + 2 * 128 * 8;
    // E4M3: [4][128] query exponents, one byte each (items i .. i+3)
    static constexpr int OFF_BAD = OFF_QEXP + (FP8 ? 4 * 128 : 0);
    static constexpr int NBAD = 16;                        // ring of the tiles' bad-block masks
    static constexpr int OFF_BAR = OFF_BAD + NBAD * 4;
    static constexpr int NBAR = 2 * NSK + 2 * NSV + 6 + 3 + 2 * NST;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;    // TMEM address, share start
    static constexpr int USED = OFF_MISC + 64;
    static constexpr int SLACK = USED + 1024 <= 227 * 1024 ? 1024 : 0;  // else the base must be aligned (checked)
    static constexpr int SMEM = USED + SLACK;
    static constexpr int NWIDEN = FP8 ? 4 : 0;
    static constexpr int W_LOAD = 8, W_MMA = 9, W_WIDEN = 12;  // warps 0-7: softmax; 10 and 11 only fill the warpgroup
    static constexpr int NT = (12 + NWIDEN) * 32;
    static constexpr uint32_t COL_O = 2 * KT;
    static constexpr uint32_t OP_ARRIVALS = FP8 ? NWIDEN * 32 : 1;  // arrivals that fill a Q, K or V tile
    // E4M3: P is kept 2^7 times larger, so that f16 holds weights down to
    // 2^-31 of the largest (and up to 2^(7 + 8) before the maximum moves)
    static constexpr float PBIAS = FP8 ? 7.f : 0.f;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(COL_O + 2 * D <= 512, "TMEM columns");
    static_assert(NSK + 2 < NBAD && (NST == 0 || NST / 2 + NSK + 3 < NBAD), "bad-block ring");
};

struct TreeWs {
    float *o;    // [2 kMaxCtas][128][D] normalised partial outputs
    float *lse;  // [2 kMaxCtas][128] log2-sum-exp
    int4 *desc;  // [kMaxCtas]: (first q row, rows, kv head, pieces) of the cut segment that begins in CTA g; pieces 0: none
};

// A sequence of the batch.
struct Seq {
    int q0, T, P;        // first row, drafts (0 if its metadata is bad), prefix
    int nmt, U;          // row tiles; line units of a segment
    PA_DEVICE int units(int Hkv) const { return Hkv * nmt * U; }
};

template <class C>
PA_DEVICE Seq load_seq(const TreeArgs &a, int b, bool flag) {
    Seq s;
    s.q0 = a.cu_q[b];
    const int64_t q1 = a.cu_q[b + 1], T = q1 - s.q0;
    s.P = a.prefix_lens[b];
    s.T = (int)T;
    if (s.q0 < 0 || T < 0 || T > a.max_q_len || q1 > a.total_q || s.P < 0 || s.P + T > (int64_t)a.max_blocks * 16) {
        if (flag) flag_error(a.err, PA_DEVERR_BAD_LEN);
        s.T = 0;
        s.P = 0;
    }
    s.nmt = (s.T + C::QPOS - 1) / C::QPOS;
    s.U = (s.P + s.T + C::KT - 1) / C::KT + kSegCost;
    return s;
}

// Key tiles [j0, j1) of one segment.
struct Item {
    int b, kvh, q0, T, P, L;   // q0: first row of the row tile; T: drafts of the sequence
    int nrows;                 // accumulator rows in use
    int j0, j1, nt;            // nt: key tiles of the segment
    int r0;                    // first draft of the row tile
};

// Walks a CTA's share of the line.
template <class C>
struct Walk {
    int64_t pos, end, base;  // base: line position of sequence b
    int64_t S;
    int b;
    Seq s;

    PA_DEVICE void start(const TreeArgs &a, int64_t pos_, int64_t end_, int64_t S_, int b0, int64_t base0) {
        pos = pos_, end = end_, S = S_, b = b0, base = base0;
        if (pos < end) s = load_seq<C>(a, b, false);
    }
    PA_DEVICE bool next(const TreeArgs &a, Item &it) {
        while (pos < end) {
            int off = (int)min(pos - base, (int64_t)INT32_MAX);
            const int units = s.units(a.Hkv);
            if (pos - base >= units) {
                base += units;
                s = load_seq<C>(a, ++b, false);
                continue;
            }
            const int seg = off / s.U, r = off - seg * s.U;
            const int64_t seg0 = pos - r;
            const int stop = (int)min((int64_t)s.U, end - seg0);
            it.j0 = max(r - kSegCost, 0);
            it.j1 = stop - kSegCost;
            pos = seg0 + stop;
            if (it.j1 <= it.j0) continue;
            it.b = b;
            it.kvh = seg / s.nmt;
            const int mt = seg - it.kvh * s.nmt;
            it.r0 = mt * C::QPOS;
            it.q0 = s.q0 + it.r0;
            it.T = s.T;
            it.P = s.P;
            it.L = s.P + s.T;
            it.nrows = min(C::QPOS, s.T - it.r0) * C::G;
            it.nt = s.U - kSegCost;
            return true;
        }
        return false;
    }
    // pieces of the segment whose item ends at pos (it began in this share):
    // the shares from the one that holds its first tile to the one that
    // holds its last
    PA_DEVICE int pieces(const Item &it) const {
        const int64_t tile0 = pos - it.j1;  // line position of the segment's first tile
        return (int)((tile0 + it.nt - 1) / S - tile0 / S) + 1;
    }
};

// One cache row's elements of a lane, widened to fp32.
template <int D, bool FP8>
PA_DEVICE void load_dims(const void *cache, int64_t row, int lane, float (&x)[D / 32]) {
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
        const int64_t at = row * D + lane * (D / 32) + e;
        if constexpr (FP8) x[e] = (float)static_cast<const __nv_fp8_e4m3 *>(cache)[at];
        else x[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(cache)[at]);
    }
}

// 16 consecutive 32-bit columns of this thread's TMEM lane.
PA_DEVICE void tmem_st16_u(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

PA_DEVICE bool not_finite(float x) { return !(fabsf(x) <= 3.4028235e38f); }

// P.V multiplies the V rows of drafts that a row does not see by zero, and
// zero times an infinity or a NaN is NaN.  So where a segment's drafts hold
// one, its affected rows are attended again, by one warp with the formula
// over the visible keys alone.  Does any V row of the sequence's drafts hold
// a value that is not finite (the kv head's)?
template <class C>
__device__ __noinline__ bool drafts_not_finite(const TreeArgs &a, const Item &it, int lane) {
    bool bad = false;
    for (int t = it.P; t < it.L; ++t) {
        const int64_t blk = a.block_tables[(size_t)it.b * a.max_blocks + (t >> 4)];
        if (blk < 0 || blk >= a.num_blocks) continue;
        float v[C::D / 32];
        load_dims<C::D, C::FP8>(a.v_cache, (blk * a.Hkv + it.kvh) * 16 + (t & 15), lane, v);
#pragma unroll
        for (int e = 0; e < C::D / 32; ++e) bad |= not_finite(v[e]);
    }
    return __any_sync(kFull, bad);
}

// sum_t 2^(s_t - m) v_t over the item's visible keys, lane l's dims.
template <class C>
__device__ __noinline__ void attend_row(const TreeArgs &a, const Item &it, int r, uint64_t bits, float m, int lane,
                                        float (&acc)[C::D / 32]) {
    constexpr int E = C::D / 32;
    float q[E];
    load_dims<C::D, false>(a.q, (int64_t)(it.q0 + r / C::G) * a.Hq + it.kvh * C::G + r % C::G, lane, q);
    const float sl2 = a.scale * kLog2e * (C::FP8 ? a.k_scale[it.kvh] : 1.f);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int t = it.j0 * C::KT; t < min(it.j1 * C::KT, it.L); ++t) {
        if (t >= it.P && !((bits >> (t - it.P)) & 1)) continue;
        const int64_t blk = a.block_tables[(size_t)it.b * a.max_blocks + (t >> 4)];
        if (blk < 0 || blk >= a.num_blocks) continue;
        const int64_t row = (blk * a.Hkv + it.kvh) * 16 + (t & 15);
        float k[E], v[E], s = 0.f;
        load_dims<C::D, C::FP8>(a.k_cache, row, lane, k);
        load_dims<C::D, C::FP8>(a.v_cache, row, lane, v);
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
        const float p = ex2(fmaf(s, sl2, -m));
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(p, v[e], acc[e]);
    }
}

template <class C>
__global__ void __launch_bounds__(C::NT, 1)
    tree_kernel(const TreeArgs a, const TreeWs ws, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmQ) {
    constexpr int D = C::D, G = C::G, KT = C::KT, NSK = C::NSK, NSV = C::NSV, NST = C::NST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *sQ = smem + C::OFF_Q, *sK = smem + C::OFF_K, *sV = smem + C::OFF_V, *sC = smem + C::OFF_C;
    float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    int8_t *qexp = reinterpret_cast<int8_t *>(smem + C::OFF_QEXP);
    volatile uint32_t *badmask = reinterpret_cast<uint32_t *>(smem + C::OFF_BAD);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *kfull = bars, *kempty = kfull + NSK, *vfull = kempty + NSK, *vempty = vfull + NSV;
    uint64_t *sfull = vempty + NSV, *pfull = sfull + 2, *odone = pfull + 2;
    uint64_t *qfull = odone + 2, *qempty = qfull + 1, *mma_done = qempty + 1;
    uint64_t *cfull = mma_done + 1, *cempty = cfull + NST;  // E4M3: staging ring of codes
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    int *s_b0 = reinterpret_cast<int *>(smem + C::OFF_MISC + 4);
    int64_t *s_base = reinterpret_cast<int64_t *>(smem + C::OFF_MISC + 8);  // base of b0; share size; total
    // scan scratch: in the (m, l) area, which is not in use yet
    int64_t *scan = reinterpret_cast<int64_t *>(smem + C::OFF_ML);

    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    pdl_trigger();
    if (C::SLACK == 0 && smem != smem_raw) {  // (uniform per launch)
        if (tid == 0) flag_error(a.err, PA_DEVERR_LAYOUT);
        pdl_wait();
        if (tid == 0) ws.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    if (w == C::W_MMA) tmem_alloc(tmem_slot, 512);
    if (tid == C::W_LOAD * 32) {
        for (int i = 0; i < NSK; ++i) {
            mbar_init(&kfull[i], C::OP_ARRIVALS);
            mbar_init(&kempty[i], 1);
        }
        for (int i = 0; i < NSV; ++i) {
            mbar_init(&vfull[i], C::OP_ARRIVALS);
            mbar_init(&vempty[i], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&pfull[s], 128);
            mbar_init(&odone[s], 1);
        }
        mbar_init(qfull, C::OP_ARRIVALS);
        mbar_init(qempty, 1);
        mbar_init(mma_done, 1);
        for (int i = 0; i < NST; ++i) {
            mbar_init(&cfull[i], 1);
            mbar_init(&cempty[i], C::NWIDEN * 32);
        }
        fence_mbar_init();
    }
    pdl_wait();
    const uint64_t deadline = wait_deadline();  // shared by every wait of this launch

    // ---- the share of this CTA: a scan over the sequences' line units
    {
        const int per = (a.B + C::NT - 1) / C::NT, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) mine += load_seq<C>(a, b, blockIdx.x == 0).units(a.Hkv);
        int64_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scan[w] = x;
        __syncthreads();
        int64_t before = x - mine, total = 0;
#pragma unroll
        for (int i = 0; i < C::NT / 32; ++i) {
            if (i < w) before += scan[i];
            total += scan[i];
        }
        const int64_t S = max((total + gridDim.x - 1) / (int64_t)gridDim.x, (int64_t)1);
        const int64_t pos = (int64_t)blockIdx.x * S;
        if (pos >= before && pos < before + mine) {  // one thread at most
            int64_t at = before;
            int b = b0;
            for (;; ++b) {
                const int u = load_seq<C>(a, b, false).units(a.Hkv);
                if (pos < at + u) break;
                at += u;
            }
            *s_b0 = b;
            s_base[0] = at;
        }
        if (tid == 0) {
            s_base[1] = S;
            s_base[2] = total;
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Walk<C> walk;
    {
        const int64_t S = s_base[1], total = s_base[2], pos = min((int64_t)blockIdx.x * S, total);
        walk.start(a, pos, min(pos + S, total), S, *s_b0, s_base[0]);
    }
    __syncthreads();  // the scan scratch is free
    // ok turns false at the first wait past the deadline; after that a role
    // issues no further wait: the loader, the MMA and the widening warps stop,
    // the softmax warps only keep their barriers in step
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        ok = ok && mbar_wait(bar, parity, deadline);
        return ok;
    };
    auto wait_all = [&](uint64_t *bar, uint32_t parity) {
        ok = ok && mbar_wait(bar, parity, deadline);
        ok = __all_sync(kFull, ok);
        return ok;
    };
    Item it;
    if (w == C::W_LOAD) {
        // ---- K tile n+1, then V tile n (the order of their use), across the
        // items of the share; a window of 32 block-table entries in registers
        const int32_t *bt = nullptr;
        int win0 = 0, went = 0, nblk = 0;
        auto open = [&](const Item &i) {
            bt = a.block_tables + (size_t)i.b * a.max_blocks;
            nblk = (i.L + 15) >> 4;
            win0 = i.j0 * C::BPT;
            went = bt[min(win0 + lane, nblk - 1)];
        };
        auto tile_row = [&](const Item &i, int j, int n) -> int64_t {  // lanes 0..7: cache row of the tile's block
            const int jb = j * C::BPT;
            if (jb + C::BPT > win0 + 32) {
                win0 = jb;
                went = bt[min(win0 + lane, nblk - 1)];
            }
            int phys = __shfl_sync(kFull, went, (min(jb + lane % C::BPT, nblk - 1) - win0) & 31);
            const bool bad = phys < 0 || phys >= a.num_blocks;  // its keys are masked
            const uint32_t m = __ballot_sync(kFull, bad && lane < C::BPT);
            if (m) {
                if (lane == 0) flag_error(a.err, PA_DEVERR_BAD_BLOCK);
                if (bad) phys = 0;
            }
            if (lane == 0) badmask[n % C::NBAD] = m;
            return ((int64_t)phys * a.Hkv + i.kvh) * 16;
        };
        int kn = 0, vn = 0, cn = 0;  // tiles issued
        auto fill = [&](int kv, int64_t row) {
            if constexpr (!C::FP8) {
                const int ns = kv ? NSV : NSK, n = kv ? vn : kn, sl = n % ns;
                if (n >= ns && !wait(kv ? &vempty[sl] : &kempty[sl], (n / ns - 1) & 1)) return false;
                (kv ? vn : kn)++;
                uint64_t *full = kv ? &vfull[sl] : &kfull[sl];
                if (lane == 0) mbar_arrive_expect_tx(full, C::TILE);
                __syncwarp();
                if (lane < C::BPT) {
                    uint8_t *dst = (kv ? sV : sK) + sl * C::TILE + lane * 16 * 128;
#pragma unroll
                    for (int at = 0; at < C::NATOM; ++at)
                        tma_load_2d(dst + at * C::ATOM, kv ? &tmV : &tmK, at * 64, (int)row, full);
                }
            } else {
                const int sl = cn % NST;
                if (cn >= NST && !wait(&cempty[sl], (cn / NST - 1) & 1)) return false;
                ++cn;
                if (lane == 0) mbar_arrive_expect_tx(&cfull[sl], C::CODES);
                __syncwarp();
                if (lane < C::BPT)
                    tma_load_2d(sC + sl * C::CODES + lane * 16 * D, kv ? &tmV : &tmK, 0, (int)row, &cfull[sl]);
            }
            __syncwarp();
            return true;
        };
        int n = 0;
        int64_t vrow = -1;
        bool go = walk.next(a, it);
        while (go && ok) {
            open(it);
            for (int j = it.j0; j < it.j1 && ok; ++j, ++n) {
                const int64_t row = tile_row(it, j, n);
                if (!fill(0, row)) break;
                if (n > 0 && !fill(1, vrow)) break;
                vrow = row;
            }
            go = ok && walk.next(a, it);
        }
        if (ok && n > 0) fill(1, vrow);
        if (!ok) {  // the last copy of every slot may be in flight: wait for it, with a short fresh budget
            const uint64_t dd = drain_deadline();
            if constexpr (!C::FP8) {
                for (int sl = 0; sl < NSK; ++sl)
                    if (kn > sl) mbar_wait(&kfull[sl], ((kn - 1 - sl) / NSK) & 1, dd);
                for (int sl = 0; sl < NSV; ++sl)
                    if (vn > sl) mbar_wait(&vfull[sl], ((vn - 1 - sl) / NSV) & 1, dd);
            } else {
                for (int sl = 0; sl < NST; ++sl)
                    if (cn > sl) mbar_wait(&cfull[sl], ((cn - 1 - sl) / NST) & 1, dd);
            }
            __syncwarp();
        }
    } else if (w == C::W_MMA) {
        constexpr uint32_t idS = idesc_f16kind_f32(128, KT, false, !C::FP8);
        constexpr uint32_t idO = idesc_f16kind_f32(128, D, true, !C::FP8);
        int n = 0, item = 0;     // tile about to get its scores; items whose query tile was requested
        bool q_flying = false;
        auto load_q = [&](const Item &i) {  // bf16: one 3-D box per 64-column atom
            if constexpr (!C::FP8) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(qfull, C::TILE);
#pragma unroll
                    for (int at = 0; at < C::NATOM; ++at)
                        tma_load_3d(sQ + at * C::ATOM, &tmQ, at * 64, i.kvh * G, i.q0, qfull);
                }
                __syncwarp();
                q_flying = true;
            }
        };
        auto scores = [&](int nn, bool last) {  // S(nn) = Q K^T, whose K tile and query tile have landed
            if (lane == 0) {
                tc_fence_after();
                const uint32_t q0 = smem_addr(sQ), k0 = smem_addr(sK + nn % NSK * C::TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_mma_bf16(tmem + (nn & 1) * KT, smem_desc_sw128(q0 + (kk / 4) * C::ATOM + (kk % 4) * 32, 16, 1024),
                                smem_desc_sw128(k0 + (kk / 4) * C::ATOM + (kk % 4) * 32, 16, 1024), idS, kk > 0);
                tc_commit(&sfull[nn & 1]);
                tc_commit(&kempty[nn % NSK]);
                if (last) tc_commit(qempty);
            }
            __syncwarp();
        };
        auto s_ready = [&](int nn) {  // its K tile has landed, its buffer is free (P(nn-2).V complete)
            return wait(&kfull[nn % NSK], (nn / NSK) & 1) && (nn < 2 || wait(&odone[nn & 1], ((nn >> 1) - 1) & 1));
        };
        auto pv = [&](int nn, int kv0, int L, bool first) {  // O += P(nn) V(nn)
            const int sl = nn % NSV;
            if (!wait(&vfull[sl], (nn / NSV) & 1)) return;
            if constexpr (!C::FP8) {  // rows past the end or of bad blocks: zero them before they meet P
                const uint32_t bad = badmask[nn % C::NBAD];
                if (kv0 + KT > L || bad) {
                    uint8_t *vt = sV + sl * C::TILE;
                    for (int r = lane; r < KT; r += 32)
                        if (kv0 + r >= L || ((bad >> (r >> 4)) & 1))
#pragma unroll
                            for (int at = 0; at < C::NATOM; ++at)
#pragma unroll
                                for (int cc = 0; cc < 8; ++cc)
                                    *reinterpret_cast<uint4 *>(vt + at * C::ATOM + r * 128 + cc * 16) =
                                        make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
            if (!wait(&pfull[nn & 1], (nn >> 1) & 1)) return;
            if (lane == 0) {
                tc_fence_after();
                const uint32_t v0 = smem_addr(sV + sl * C::TILE);
#pragma unroll
                for (int kk = 0; kk < KT / 16; ++kk)
                    tc_mma_bf16_tmem_a(tmem + C::COL_O + (nn & 1) * D, tmem + (nn & 1) * KT + kk * 8,
                                       smem_desc_sw128(v0 + kk * 16 * 128, C::ATOM, 1024), idO, !first || kk > 0);
                tc_commit(&odone[nn & 1]);
                tc_commit(&vempty[sl]);
            }
            __syncwarp();
        };
        bool go = walk.next(a, it);
        if (go) load_q(it);
        while (go && ok) {
            const Item cur = it;
            const int cnt = cur.j1 - cur.j0;
            bool more = false;
            if (!wait(qfull, item & 1)) break;
            q_flying = false;
            ++item;
            if (!s_ready(n)) break;
            scores(n, cnt == 1);
            for (int j = 0; j < cnt && ok; ++j) {
                if (j + 1 < cnt) {
                    if (!s_ready(n + 1)) break;
                    scores(n + 1, j + 2 == cnt);
                }
                if (j + 2 >= cnt && (cnt == 1 || j + 2 == cnt)) {  // all scores issued: fetch the next query tile
                    more = walk.next(a, it);
                    if (!C::FP8 && more) {
                        if (!wait(qempty, (item - 1) & 1)) break;
                        load_q(it);
                    }
                }
                pv(n, (cur.j0 + j) * KT, cur.L, j < 2);
                ++n;
            }
            go = more;
        }
        // every MMA of this CTA has completed before TMEM is released, and
        // the query copy has landed
        if (lane == 0) tc_commit(mma_done);
        __syncwarp();
        if (!ok && q_flying) mbar_wait(qfull, item & 1, drain_deadline());
        const bool done = mbar_wait(mma_done, 0, ok ? deadline : drain_deadline());
        ok = __all_sync(kFull, ok && done);
    } else if (w >= C::W_WIDEN) {
      if constexpr (C::FP8) {
        // ---- E4M3: thread ct widens key row ct of each staged tile into its
        // f16 operand tile, and scales query row ct
        const int ct = tid - C::W_WIDEN * 32;
        int kn = 0, vn = 0, cn = 0, item = 0;
        auto widen = [&](int kv, int kv0, int L, int n) {
            const int ns = kv ? NSV : NSK, m = kv ? vn : kn, sl = m % ns, cs = cn % NST;
            if (!wait(&cfull[cs], (cn / NST) & 1)) return false;
            if (m >= ns && !wait(kv ? &vempty[sl] : &kempty[sl], (m / ns - 1) & 1)) return false;
            (kv ? vn : kn)++;
            ++cn;
            uint8_t *tile = (kv ? sV : sK) + sl * C::TILE;
            const uint8_t *codes = sC + cs * C::CODES + ct * D;
            const bool live = kv0 + ct < L && !((badmask[n % C::NBAD] >> (ct >> 4)) & 1);
            uint4 src[D / 16];
#pragma unroll
            for (int u = 0; u < D / 16; ++u) {  // the codes' rows are swizzled too: conflict-free columns
                const int ch = D == 128 ? (u ^ (ct & 7)) : (u ^ ((ct >> 1) & 3));
                src[u] = live ? *reinterpret_cast<const uint4 *>(codes + 16 * ch) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < D / 16; ++u) {
                const uint32_t wd[4] = {src[u].x, src[u].y, src[u].z, src[u].w};
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[2 * e] = e4m3x2_to_h2(wd[e]);
                    h[2 * e + 1] = e4m3x2_to_h2(wd[e] >> 16);
                }
#pragma unroll
                for (int hc = 0; hc < 2; ++hc) {
                    const int ch = 2 * u + hc, at = ch / 8, cc = ch % 8;
                    *reinterpret_cast<uint4 *>(tile + at * C::ATOM + ct * 128 + ((cc ^ (ct & 7)) * 16)) =
                        make_uint4(h[4 * hc], h[4 * hc + 1], h[4 * hc + 2], h[4 * hc + 3]);
                }
            }
            mbar_arrive(&cempty[cs]);
            fence_proxy_async_smem();
            mbar_arrive(kv ? &vfull[sl] : &kfull[sl]);
            return true;
        };
        auto query = [&](const Item &i) {  // f16(q 2^e), e per row: its largest magnitude in [2^14, 2^15)
            const bool live = ct < i.nrows;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const __nv_bfloat16 *>(a.q) + ((size_t)(i.q0 + ct / G) * a.Hq + (size_t)i.kvh * G + ct % G) * D);
            uint4 v[D / 8];
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                v[k] = live ? src[k] : make_uint4(0, 0, 0, 0);
                const uint32_t wd[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = bf16x2_to_float2(wd[e]);
                    amax = fmax3(amax, fabsf(f.x), fabsf(f.y));
                }
            }
            int ex = 0;
            if (amax > 0.f) ex = min(max(14 - ((int)((__float_as_uint(amax) >> 23) & 0xff) - 127), -100), 100);
            const float qs = __uint_as_float((uint32_t)(127 + ex) << 23);
            if (item > 0 && !wait(qempty, (item - 1) & 1)) return false;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const uint32_t wd[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = bf16x2_to_float2(wd[e]);
                    const __half2 hh = __floats2half2_rn(f.x * qs, f.y * qs);
                    h[e] = *reinterpret_cast<const uint32_t *>(&hh);
                }
                const int at = k / 8, cc = k % 8;
                *reinterpret_cast<uint4 *>(sQ + at * C::ATOM + ct * 128 + ((cc ^ (ct & 7)) * 16)) =
                    make_uint4(h[0], h[1], h[2], h[3]);
            }
            qexp[(item & 3) * 128 + ct] = (int8_t)ex;
            ++item;
            fence_proxy_async_smem();
            mbar_arrive(qfull);
            return true;
        };
        // K tile n+1 before V tile n, as the loader; an item's query tile
        // before the first V that follows its first K
        int n = 0, vkv0 = 0, vL = 0;
        while (ok && walk.next(a, it)) {
            for (int j = it.j0; j < it.j1 && ok; ++j, ++n) {
                if (!widen(0, j * KT, it.L, n)) break;
                if (n > 0 && !widen(1, vkv0, vL, n - 1)) break;
                if (j == it.j0 && !query(it)) break;
                vkv0 = j * KT;
                vL = it.L;
            }
        }
        if (ok && n > 0) widen(1, vkv0, vL, n - 1);
      }
    } else if (w < 8) {
        // ---- softmax: warpgroup g takes the tiles n with n % 2 == g; thread
        // = row r of the row tile
        const int g = w >> 2, r = (w & 3) * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)((w & 3) * 32) << 16);
        const uint32_t scol = g * KT, ocol = C::COL_O + g * D;
        int n = 0, item = 0;
        int4 desc = make_int4(0, 0, 0, 0);
        while (walk.next(a, it)) {
            const int cnt = it.j1 - it.j0;
            const bool warp_live = (w & 3) * 32 < it.nrows, row_live = r < it.nrows;
            uint64_t bits = 0;
            if (row_live) {
                bits = a.mask[it.q0 + r / G];
                if (it.T < 64) bits &= (1ull << it.T) - 1;
            }
            float sl2 = a.scale * kLog2e * (C::FP8 ? a.k_scale[it.kvh] : 1.f);
            const float vs = C::FP8 ? a.v_scale[it.kvh] : 1.f;
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            bool have = false;
            for (int j = (n ^ g) & 1; j < cnt; j += 2) {
                const int nn = n + j, kv0 = (it.j0 + j) * KT;
                const bool landed = wait_all(&sfull[g], (nn >> 1) & 1);
                if (landed && warp_live) {
                    tc_fence_after();
                    if (C::FP8 && !have) sl2 *= __uint_as_float((uint32_t)(127 - qexp[(item & 3) * 128 + r]) << 23);
                    // the keys this row may see, where the tile is not all prefix
                    const uint32_t bad = badmask[nn % C::NBAD];
                    const bool masked = kv0 + KT > it.P || bad;
                    auto visible = [&](int q) -> uint32_t {  // keys kv0 + 32 q + [0, 32)
                        const int rel = kv0 + 32 * q - it.P;  // draft of the first one
                        uint32_t v = rel <= -32  ? kFull
                                     : rel >= 64 ? 0u
                                     : rel < 0   ? (uint32_t)((bits << -rel) | ((1ull << -rel) - 1))
                                                 : (uint32_t)(bits >> rel);
                        if ((bad >> (2 * q)) & 1) v &= 0xffff0000u;
                        if ((bad >> (2 * q + 1)) & 1) v &= 0x0000ffffu;
                        return v;
                    };
                    constexpr int NH = 4, HC = KT / NH;  // the scores are read twice, HC in registers at a time
                    float sv[HC];
                    auto load = [&](int h) {
#pragma unroll
                        for (int q = 0; q < HC / 32; ++q) {
                            float t32[32];
                            tmem_ld32(lane_base + scol + h * HC + 32 * q, t32);
#pragma unroll
                            for (int e = 0; e < 32; ++e) sv[32 * q + e] = t32[e];
                        }
                        tmem_wait_ld();
                        if (masked) {
#pragma unroll
                            for (int q = 0; q < HC / 32; ++q) {
                                const uint32_t v = visible(h * (HC / 32) + q);
#pragma unroll
                                for (int e = 0; e < 32; ++e) sv[32 * q + e] = (v >> e) & 1 ? sv[32 * q + e] : -INFINITY;
                            }
                        }
                    };
                    float mx = -INFINITY;
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        load(h);
#pragma unroll
                        for (int e = 0; e < HC; e += 2) mx = fmax3(mx, sv[e], sv[e + 1]);
                    }
                    const float mt = mx * sl2;  // (the scale is positive)
                    const bool rescale = mt > m + kRescaleThreshold;
                    float alpha = 1.f;
                    if (rescale) {
                        alpha = ex2(m - mt);  // m = -inf: 0
                        m = mt;
                        l2 = make_float2(l2.x * alpha, l2.y * alpha);
                    }
                    const float nb = (m == -INFINITY ? 0.f : -m) + C::PBIAS;
                    const float2 sc2 = make_float2(sl2, sl2), nb2 = make_float2(nb, nb);
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        if (NH > 1) load(h);
#pragma unroll
                        for (int q = 0; q < HC / 32; ++q) {
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                const float2 x = ffma2(make_float2(sv[32 * q + e], sv[32 * q + e + 1]), sc2, nb2);
                                const float2 p = make_float2(ex2(x.x), ex2(x.y));
                                l2 = fadd2(l2, p);
                                if constexpr (C::FP8) {
                                    const __half2 hh = __floats2half2_rn(p.x, p.y);
                                    pk[e / 2] = *reinterpret_cast<const uint32_t *>(&hh);
                                } else {
                                    const __nv_bfloat162 bb = __floats2bfloat162_rn(p.x, p.y);
                                    pk[e / 2] = *reinterpret_cast<const uint32_t *>(&bb);
                                }
                            }
                            // P over score columns that this thread has read
                            tmem_st16_u(lane_base + scol + 16 * (h * (HC / 32) + q), pk);
                        }
                    }
                    // O holds P.V up to this warpgroup's previous tile, complete
                    // (this tile's scores were issued after it)
                    if (have && __any_sync(kFull, rescale)) {
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            float o[32];
                            tmem_ld32(lane_base + ocol + 32 * q, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= alpha;
                            tmem_st32(lane_base + ocol + 32 * q, o);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    have = true;
                }
                mbar_arrive(&pfull[g]);
            }
            // ---- join the two accumulators: warpgroup g writes columns
            // [g D/2, (g+1) D/2) of every row
            ml[g * 128 + r] = make_float2(m, l2.x + l2.y);
            named_bar_sync(kEpiBar, 256);
            const float2 ml0 = ml[r], ml1 = ml[128 + r];
            const int last = n + cnt - 1;  // its stream's last tile; the other stream's is last - 1
            bool landed = wait_all(&odone[last & 1], (last >> 1) & 1);
            if (cnt > 1) landed = wait_all(&odone[(last - 1) & 1], ((last - 1) >> 1) & 1);
            const bool one = cnt == 1;  // a single tile: one accumulator
            const float M = fmaxf(ml0.x, ml1.x);
            const float f0 = ml0.x == -INFINITY ? 0.f : ex2(ml0.x - M), f1 = ml1.x == -INFINITY ? 0.f : ex2(ml1.x - M);
            const float l = ml0.y * f0 + ml1.y * f1;
            const float inv = (l > 0.f ? 1.f / l : l == l ? 0.f : l) * vs;
            const bool whole = it.j0 == 0 && it.j1 == it.nt;
            const size_t grow = ((size_t)(it.q0 + r / G) * a.Hq + (size_t)it.kvh * G + r % G);
            const int slot = blockIdx.x * 2 + (it.j0 == 0 ? 1 : 0);
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + grow * D + g * (D / 2);
            float *wo = ws.o + ((size_t)slot * 128 + r) * D + g * (D / 2);
            if (landed && warp_live) {
                tc_fence_after();
                bool odd = false;
#pragma unroll 1
                for (int q = 0; q < D / 64; ++q) {
                    float o[32], o1[32];
                    const uint32_t col = lane_base + C::COL_O + g * (D / 2) + 32 * q;
                    tmem_ld32(col + (one ? (last & 1) * D : 0), o);
                    if (!one) tmem_ld32(col + D, o1);
                    tmem_wait_ld();
                    const float w0 = (one ? ((last & 1) ? f1 : f0) : f0) * inv, w1 = f1 * inv;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        o[e] = l == 0.f ? 0.f : one ? o[e] * w0 : fmaf(o1[e], w1, o[e] * w0);
                        odd |= not_finite(o[e]);
                    }
                    if (!row_live) continue;
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t wd[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const __nv_bfloat162 bb = __floats2bfloat162_rn(o[e + 2 * u], o[e + 2 * u + 1]);
                                wd[u] = *reinterpret_cast<const uint32_t *>(&bb);
                            }
                            *reinterpret_cast<uint4 *>(dst + 32 * q + e) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(wo + 32 * q + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (!whole && row_live && g == 0)
                    ws.lse[slot * 128 + r] = l > 0.f ? M + lg2(l) - C::PBIAS : l == l ? -INFINITY : l;
                // rows that an unseen draft's V spoilt
                uint32_t todo = __ballot_sync(kFull, odd && row_live && l > 0.f && l <= 3.4028235e38f);
                if (todo && it.j1 * KT > it.P && drafts_not_finite<C>(a, it, lane)) {
                    while (todo) {
                        const int rl = __ffs(todo) - 1;
                        todo &= todo - 1;
                        const int rr = (w & 3) * 32 + rl;
                        float acc[D / 32];
                        attend_row<C>(a, it, rr, __shfl_sync(kFull, bits, rl), __shfl_sync(kFull, M, rl) - C::PBIAS, lane, acc);
                        const float iv = __shfl_sync(kFull, inv, rl);
                        if ((lane * (D / 32)) / (D / 2) == g) {
                            const size_t gr = (size_t)(it.q0 + rr / G) * a.Hq + (size_t)it.kvh * G + rr % G;
#pragma unroll
                            for (int e = 0; e < D / 32; ++e) {
                                const int d = lane * (D / 32) + e;
                                if (whole) static_cast<__nv_bfloat16 *>(a.out)[gr * D + d] = __float2bfloat16_rn(acc[e] * iv);
                                else ws.o[((size_t)slot * 128 + rr) * D + d] = acc[e] * iv;
                            }
                        }
                    }
                }
            }
            tc_fence_before();
            named_bar_sync(kEpiBar, 256);  // both accumulators and (m, l) are read
            n += cnt;
            ++item;
            if (!whole && it.j0 == 0) desc = make_int4(it.q0, it.nrows, it.kvh, walk.pieces(it));  // the share's last item
        }
        if (tid == 0) ws.desc[blockIdx.x] = desc;
    }
    if (!ok && lane == 0) flag_error(a.err, PA_DEVERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (w == C::W_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Log-sum-exp merge of the cut segment that begins in CTA blockIdx.x: piece 0
// in its slot 2 g + 1, the others in slot 2 (g + p) of the CTAs after it.
// One warp per row.
template <int D, int G>
__global__ void __launch_bounds__(128) tree_merge_kernel(const TreeArgs a, const TreeWs ws, int ctas) {
    constexpr int E = D / 32;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, g = blockIdx.x;
    const int4 d = ws.desc[g];
    const int np = d.w;
    if (np < 1 || g + np > ctas) return;
    for (int r = blockIdx.y * 4 + (threadIdx.x >> 5); r < d.y; r += gridDim.y * 4) {
        auto at = [&](int p) { return (size_t)(2 * (g + p) + (p == 0 ? 1 : 0)) * 128 + r; };
        float m = -INFINITY, l = 0.f;
        for (int p = lane; p < np; p += 32) m = fmaxf(m, __ldcg(ws.lse + at(p)));
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        const float mb = m == -INFINITY ? 0.f : m;
        for (int p = lane; p < np; p += 32) l += ex2(__ldcg(ws.lse + at(p)) - mb);
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
        const float inv = l > 0.f ? 1.f / l : l == l ? 0.f : l;
        float acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
        for (int p = 0; p < np; ++p) {
            const float lp = __ldcg(ws.lse + at(p)), wt = ex2(lp - mb) * inv;
            const float *src = ws.o + at(p) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = __ldcg(reinterpret_cast<const float2 *>(src + e));
                // a piece without weight (none of its keys is visible) adds nothing
                acc[e] = lp == -INFINITY ? acc[e] : fmaf(wt, v.x, acc[e]);
                acc[e + 1] = lp == -INFINITY ? acc[e + 1] : fmaf(wt, v.y, acc[e + 1]);
            }
        }
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) +
                             ((size_t)(d.x + r / G) * a.Hq + (size_t)d.z * G + r % G) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<__nv_bfloat162 *>(dst + e) = __floats2bfloat162_rn(acc[e], acc[e + 1]);
    }
}

// ---- host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// A tensor of `rank` dims (innermost first, `elem` bytes an element), boxes
// of `box`.
bool tiled_map(CUtensorMap *map, CUtensorMapDataType type, int elem, int rank, const void *base, const cuuint64_t *dims,
               const cuuint32_t *box, CUtensorMapSwizzle swizzle) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t strides[2] = {};
    cuuint64_t s = elem;
    for (int i = 0; i + 1 < rank; ++i) strides[i] = s *= dims[i];
    const cuuint32_t ones[3] = {1, 1, 1};
    return fn(map, type, rank, const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
cudaError_t run_tree(const TreeArgs &a, const TreeWs &ws, cudaStream_t st) {
    static std::mutex mu;
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            e = cudaFuncSetAttribute(tree_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    CUtensorMap tk, tv, tq = {};
    const cuuint64_t cdims[2] = {(cuuint64_t)C::D, (cuuint64_t)a.num_blocks * a.Hkv * 16};
    const cuuint32_t cbox[2] = {C::FP8 ? (cuuint32_t)C::D : 64u, 16};
    const auto type = C::FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const auto swz = C::FP8 && C::D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    if (!tiled_map(&tk, type, C::FP8 ? 1 : 2, 2, a.k_cache, cdims, cbox, swz) ||
        !tiled_map(&tv, type, C::FP8 ? 1 : 2, 2, a.v_cache, cdims, cbox, swz))
        return cudaErrorInvalidValue;
    if (!C::FP8) {
        const cuuint64_t qdims[3] = {(cuuint64_t)C::D, (cuuint64_t)a.Hq, (cuuint64_t)a.total_q};
        const cuuint32_t qbox[3] = {64, (cuuint32_t)C::G, (cuuint32_t)C::QPOS};
        if (!tiled_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, 3, a.q, qdims, qbox, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    // a CTA per SM, fewer where the batch has fewer key tiles
    const long long tiles = (long long)a.B * a.Hkv * ((a.max_q_len + C::QPOS - 1) / C::QPOS) *
                            ((a.max_blocks + C::BPT - 1) / C::BPT + kSegCost);
    const int ctas = (int)std::min<long long>({tiles, sm_count(), kMaxCtas});
    e = launch_pdl(tree_kernel<C>, dim3(ctas), dim3(C::NT), C::SMEM, st, a, ws, tk, tv, tq);
    if (e != cudaSuccess) return e;
    return launch_pdl(tree_merge_kernel<C::D, C::G>, dim3(ctas, 8), dim3(128), 0, st, a, ws, ctas);
}

template <int D, bool FP8>
cudaError_t tree_by_group(const TreeArgs &a, const TreeWs &ws, cudaStream_t st) {
    switch (a.Hq / a.Hkv) {
        case 1: return run_tree<TCfg<D, 1, FP8>>(a, ws, st);
        case 2: return run_tree<TCfg<D, 2, FP8>>(a, ws, st);
        case 4: return run_tree<TCfg<D, 4, FP8>>(a, ws, st);
        case 8: return run_tree<TCfg<D, 8, FP8>>(a, ws, st);
        default: return cudaErrorNotSupported;
    }
}

constexpr size_t kLseBytes = 2 * kMaxCtas * 128 * sizeof(float), kDescBytes = kMaxCtas * sizeof(int4);

}  // namespace

size_t tree_ws_bytes(int D) { return kLseBytes + kDescBytes + (size_t)2 * kMaxCtas * 128 * D * sizeof(float); }

cudaError_t launch_tree(const TreeArgs &a, void *workspace, cudaStream_t st) {
    char *p = static_cast<char *>(workspace);
    const TreeWs ws{reinterpret_cast<float *>(p + kLseBytes + kDescBytes), reinterpret_cast<float *>(p),
                    reinterpret_cast<int4 *>(p + kLseBytes)};
    if (a.D == 128) return a.fp8 ? tree_by_group<128, true>(a, ws, st) : tree_by_group<128, false>(a, ws, st);
    if (a.D == 64) return a.fp8 ? tree_by_group<64, true>(a, ws, st) : tree_by_group<64, false>(a, ws, st);
    return cudaErrorNotSupported;
}

}  // namespace pa
