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
// Work split: a row tile is 128 accumulator rows = 128/G drafts x the G query
// heads of a kv head; a segment is (sequence, kv head, one or two row tiles),
// so K and V are read from HBM once per sequence (further segments, T G >
// 256, find them in L2).  The segments' key tiles (128 keys, 8 blocks) form
// one line of cost units (SEG at the head of a segment, kOne or kPair a
// tile), cut into equal contiguous shares, one per SM.  Of the segments a
// CTA meets only its first can have begun before its share and only its last
// can go on behind it, so two slots a CTA hold every partial result, whatever
// the batch; the merge kernel joins them by log-sum-exp (tree_split.h, which
// the tests compile for the host).
//
// Within a CTA the work is a line of steps, each the scores, softmax and P.V
// of one row tile and one key tile; steps alternate between two streams, each
// with its own score buffer and output accumulator in TMEM and its own softmax
// warpgroup (a thread owns a whole row of 128 scores: no exchange between
// threads).  A segment of two row tiles has one on each stream, sharing the K
// and V tiles; of one row tile the streams take the key tiles in turn, and the
// two accumulators are joined at the end.  A loader warp gathers K and V tiles
// through the block table (TMA boxes, 128-byte swizzle) into two rings; one
// thread issues the MMAs, the scores of step n+1 before P.V of step n, so that
// the tensor pipe works while the exponentials run.  P is written over its
// scores in TMEM and is the A operand of P.V, half a tile (64 keys) at a time.
// Warps whose 32 rows are all past the drafts skip the arithmetic.
// An E4M3 cache: the codes land in a staging ring and four warps widen them
// to f16 operand tiles; two more scale the query rows by a power of two into
// f16's range (which rounds components below 2^-28 of their row's largest).
// f16 and not bf16 because every code is an f16 value and P keeps three more
// bits.
// P is rounded for its product alone, to the cache's own type: both operands
// of an MMA have one type, and V in bf16 has 8 bits as well.  That is up to
// 2^-8 of a weight (f16: 2^-11); the row's sum takes the weights unrounded.
// Against 64 bits, relative to the outputs' size: 2.1e-3 to 2.3e-3, of which
// the bf16 output alone is 1.7e-3; E4M3: 1.7e-3.
//
// Bound (kernel alone, 8 kv heads, head_dim 128):
//   16 x 32701 tokens, 32 drafts (128 rows a kv head): 334 us, 2.15 GB,
//     6.4 TB/s, tensor pipe 45% -- HBM; called back to back for a second the
//     1 kW power cap lowers the clock to 1.3 GHz and a call takes 390-415 us.
//   64 x U[1,2048], 16 drafts: 66 us, 290 MB, 4.4 TB/s -- the segments, 3.5 a
//     CTA: one of a single key tile takes 3.0 us against 1.45 us for a tile in
//     a row (query tile, softmax, P.V and epilogue follow one another once),
//     and its rows fill half of a row tile.
//   E4M3, 32 x U[1,8192], U[1,64] drafts of 64 heads: 260 us -- latency: no
//     pipe is above 45% busy; a step's scores wait for the P.V that frees
//     their columns, and 16 warps leave 128 registers a thread.
// Measured and dropped: 64-key steps with two score buffers a stream (every
// MMA N = 64; E4M3 64 drafts x 8000 tokens 794 against 702 us); a part of the
// exponentials on the FMA pipe (797 against 771); a whole warp issuing the
// MMAs in step, with votes after its waits (the same time); one pass over the
// scores against the maximum so far, repeated where it moved (P of a
// whole tile in registers: spills with an E4M3 cache); registers moved between warpgroups (the calls of the rare
// path cannot be compiled so).
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"
#include "tma_map.h"
#include "tree_split.h"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units the running maximum may lag behind
constexpr int kMaxCtas = 160;              // partial-result slots: two a CTA
constexpr int kEpiBar = 1;                 // named barrier of the softmax warps
constexpr unsigned kFull = 0xffffffffu;

template <int D_, int G_, bool FP8_>
struct TCfg {
    static constexpr int D = D_, G = G_;
    static constexpr bool FP8 = FP8_;
    static constexpr int M = kTreeRows, KT = kTreeKeys, BPT = KT / 16;
    static constexpr int QPOS = M / G;             // drafts of a row tile
    static constexpr int NATOM = D / 64;           // 128-byte column atoms along D
    static constexpr int ATOM = 128 * 128;         // bytes of one atom column of a 128-row tile
    static constexpr int TILE = NATOM * ATOM;      // a Q, K or V operand tile
    // K and V tiles: 8-key groups of NATOM x 8 rows x 128 bytes, so that the
    // groups lie a uniform stride apart (as the MMA descriptors need) and a
    // block's 16 rows, both column atoms, are one 4 KB copy (head_dim 128).
    // An SM pulls 33 B a clock in 4 KB copies but 23 in 2 KB ones
    static constexpr int GROUP = NATOM * 1024;
    static constexpr int CODES = KT * D;           // a tile of E4M3 codes
    // rings: what two query tiles leave of the shared memory, so that the
    // copies in flight cover the HBM latency (an SM's share of the bandwidth
    // is ~24 B a clock).  E4M3: operand tiles and a staging ring of codes
    static constexpr int NSK = D == 128 ? (FP8 ? 2 : 3) : (FP8 ? 2 : 6);
    static constexpr int NSV = D == 128 ? (FP8 ? 1 : 2) : (FP8 ? 2 : 6);
    static constexpr int NST = FP8 ? (D == 128 ? 4 : 12) : 0;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = 2 * TILE;
    static constexpr int OFF_V = OFF_K + NSK * TILE;
    static constexpr int OFF_C = OFF_V + NSV * TILE;
    static constexpr int OFF_ML = OFF_C + NST * CODES;     // [2][128] (m, l) of the two softmax warpgroups
    static constexpr int OFF_QEXP = OFF_ML + 2 * 128 * 8;
    static constexpr int OFF_BAD = OFF_QEXP + (FP8 ? 4 * 128 : 0);  // E4M3: query exponents of 4 query tiles, a byte a row
    static constexpr int NBAD = 16;                        // ring of the key tiles' bad-block masks
    static constexpr int OFF_BAR = OFF_BAD + NBAD * 4;
    static constexpr int NBAR = 2 * NSK + 2 * NSV + 10 + 5 + 2 * NST;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;    // TMEM address, share start
    static constexpr int USED = OFF_MISC + 64;
    static constexpr int SLACK = USED + 1024 <= 227 * 1024 ? 1024 : 0;  // else the base must be aligned (checked)
    static constexpr int SMEM = USED + SLACK;
    static constexpr int NWIDEN = FP8 ? 4 : 0;
    // warps 0-7: softmax; 10 (E4M3: and 11): query tiles
    static constexpr int W_LOAD = 8, W_MMA = 9, W_QUERY = 10, W_WIDEN = 12;
    static constexpr int NT = (12 + NWIDEN) * 32;
    // line units of a segment itself (its query tile, first tile and epilogue):
    // 64 x 100 tokens take 3.0 us a segment of one tile against 1.45 us a tile
    // (bf16), 8 against 2 us (E4M3)
    static constexpr int SEG = FP8 ? kSegE4m3 : kSegBf16;
    // the next item's first K tile before this one's last V tile, or behind
    // it: widening K takes as long as a softmax, so E4M3 wants it early (64 x
    // 1000 tokens, 16 drafts: 102 against 108 us); a bf16 tile is only a copy
    // (64 x U[1,2048], 16 drafts: 72 against 69)
    static constexpr bool ACROSS = FP8;
    static constexpr uint32_t COL_O = 2 * KT;
    static constexpr uint32_t KV_ARRIVALS = FP8 ? NWIDEN * 32 : 1, Q_ARRIVALS = FP8 ? 64 : 1;  // that fill a tile
    static constexpr float OPMUL = FP8 ? 256.f : 1.f;  // E4M3: K and V operands are 2^-8 of their value (widen4)
    // E4M3: P is kept 2^7 times larger, so that f16 holds weights down to
    // 2^-31 of the largest (and up to 2^(7 + 8) before the maximum moves)
    static constexpr float PBIAS = FP8 ? 7.f : 0.f;
    static_assert(SEG <= 7 && kPair <= 3, "tree_fits() counts on it");
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(COL_O + 2 * D <= 512, "TMEM columns");
    static_assert(NSK + 3 < NBAD && NST / 2 + NSK + 3 < NBAD, "bad-block ring");
};

struct TreeWs {
    float *o;    // [2 kMaxCtas][256][D] normalised partial outputs
    float *lse;  // [2 kMaxCtas][256] log2-sum-exp
    int4 *desc;  // [kMaxCtas]: (first q row, rows, kv head, pieces) of the cut segment that begins in CTA g; pieces 0: none
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

// True in one thread of the (converged) warp.  The tensor-core and TMA
// instructions take their operands from uniform registers: behind this
// predicate the compiler knows that one thread is active, behind lane == 0 it
// wraps each of them in a loop over the active lanes' values.
PA_DEVICE bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// Has phase `parity` of `bar` completed?  (Does not suspend the thread.)
PA_DEVICE bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// The 16 rows of a block (two groups of 8, from group `g`): columns, rows,
// column atoms, groups.  No multicast.
PA_DEVICE void tma_load_4d(void *dst_smem, const CUtensorMap *map, int g, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], "
        "[%4];" ::"r"(smem_addr(dst_smem)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(g), "r"(smem_addr(bar))
        : "memory");
}

// 16 consecutive fp32 columns of this thread's TMEM lane.
PA_DEVICE void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Four E4M3 codes -> two f16x2 of 2^-8 their value: exponent and significand
// moved up by 7 and the sign by 8, which leaves the exponent 8 below f16's
// bias (subnormals included; a NaN code becomes 0x3f80).  Half of the steps
// are multiplications (x 2^7), on the FMA pipe; the conversion instruction
// shares its pipe with the exponentials.
PA_DEVICE void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    uint32_t a, b;
    asm("prmt.b32 %0, %1, 0, 0x4140;" : "=r"(a) : "r"(w));  // codes 0 and 1 as the low bytes of the halves
    asm("prmt.b32 %0, %1, 0, 0x4342;" : "=r"(b) : "r"(w));
    asm("mul.lo.u32 %0, %1, 128;" : "=r"(lo) : "r"(a));
    asm("mad.lo.u32 %0, %1, 128, %0;" : "+r"(lo) : "r"(a & 0x00800080u));
    asm("mul.lo.u32 %0, %1, 128;" : "=r"(hi) : "r"(b));
    asm("mad.lo.u32 %0, %1, 128, %0;" : "+r"(hi) : "r"(b & 0x00800080u));
}

// The same by the conversion instruction, for half of the words: that runs on
// the exponentials' pipe, which the integer forms leave idle.
PA_DEVICE void widen4_cvt(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const __half2 s = __floats2half2_rn(0x1p-8f, 0x1p-8f);  // (exact: the smallest code is 2^-9)
    const uint32_t l = e4m3x2_to_h2(w), h = e4m3x2_to_h2(w >> 16);
    const __half2 a = __hmul2(*reinterpret_cast<const __half2 *>(&l), s), b = __hmul2(*reinterpret_cast<const __half2 *>(&h), s);
    lo = *reinterpret_cast<const uint32_t *>(&a);
    hi = *reinterpret_cast<const uint32_t *>(&b);
}

// Chunks 2u and 2u + 1 (8 f16 each) of a swizzled operand row.
template <class C>
PA_DEVICE void store_chunks(uint8_t *row, int u, int r, const uint32_t (&h)[8]) {
#pragma unroll
    for (int hc = 0; hc < 2; ++hc) {
        const int ch = 2 * u + hc, at = ch / 8, cc = ch % 8;
        *reinterpret_cast<uint4 *>(row + at * 1024 + ((cc ^ (r & 7)) * 16)) =
            make_uint4(h[4 * hc], h[4 * hc + 1], h[4 * hc + 2], h[4 * hc + 3]);
    }
}

// P.V multiplies the V rows of drafts that a row does not see by zero, and
// zero times an infinity or a NaN is NaN.  So where a segment's drafts hold
// one, its affected rows are attended again, by one warp with the formula
// over the visible keys alone.  Does any V row of the sequence's drafts hold
// a value that is not finite (the kv head's)?
template <class C>
__device__ __noinline__ bool drafts_not_finite(const TreeArgs &a, const Item &it, int lane) {
    bool bad = false;
#pragma unroll 1
    for (int t = it.P + lane; t < it.L; t += 32) {  // a draft a lane
        const int64_t blk = a.block_tables[(size_t)it.b * a.max_blocks + (t >> 4)];
        if (blk < 0 || blk >= a.num_blocks) continue;
        const int64_t row = (blk * a.Hkv + it.kvh) * 16 + (t & 15);
        constexpr int E = C::FP8 ? 1 : 2;
        const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.v_cache) + row * C::D * E);
#pragma unroll
        for (int i = 0; i < C::D * E / 16; ++i) {
            const uint4 x = v[i];
            const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (C::FP8) {  // a code of seven ones
                    bad |= (((wd[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                } else {  // an exponent of eight ones
                    bad |= (wd[e] & 0x7f80u) == 0x7f80u || (wd[e] & 0x7f800000u) == 0x7f800000u;
                }
            }
        }
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
#pragma unroll 1
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
    tree_kernel(const __grid_constant__ TreeArgs a, const TreeWs ws, const __grid_constant__ CUtensorMap tmK,
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
    // per stream: scores; P of keys 0-63 (+ 2: of 64-127); P.V of keys 0-63; P.V whole
    uint64_t *sfull = vempty + NSV, *pfull = sfull + 2, *ohalf = pfull + 4, *odone = ohalf + 2;
    uint64_t *qfull = odone + 2, *qempty = qfull + 2, *mma_done = qempty + 2;
    uint64_t *cfull = mma_done + 1, *cempty = cfull + NST;  // E4M3: staging ring of codes
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    int *s_b0 = reinterpret_cast<int *>(smem + C::OFF_MISC + 4);
    int *s_base = reinterpret_cast<int *>(smem + C::OFF_MISC + 8);  // base of b0; share size; total
    // scan scratch: in the (m, l) area, which is not in use yet
    int *scan = reinterpret_cast<int *>(smem + C::OFF_ML);

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
            mbar_init(&kfull[i], C::KV_ARRIVALS);
            mbar_init(&kempty[i], 1);
        }
        for (int i = 0; i < NSV; ++i) {
            mbar_init(&vfull[i], C::KV_ARRIVALS);
            mbar_init(&vempty[i], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&pfull[s], 128);
            mbar_init(&pfull[2 + s], 128);
            mbar_init(&ohalf[s], 1);
            mbar_init(&odone[s], 1);
            mbar_init(&qfull[s], C::Q_ARRIVALS);
            mbar_init(&qempty[s], 1);
        }
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
        int mine = 0;  // (the whole line has less than 2^31 units: checked on the host)
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const Seq q = make_seq<C>(a, load_raw(a, b));
            if (q.bad && blockIdx.x == 0) flag_error(a.err, PA_DEVERR_BAD_LEN);
            mine += q.units_head(C::SEG) * a.Hkv;
        }
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scan[w] = x;
        __syncthreads();
        int before = x - mine, total = 0;
#pragma unroll
        for (int i = 0; i < C::NT / 32; ++i) {
            if (i < w) before += scan[i];
            total += scan[i];
        }
        const int S = tree_share(total, gridDim.x);
        const int64_t pos = (int64_t)blockIdx.x * S;  // (may lie past the line)
        if (pos >= before && pos < before + mine) {  // one thread at most
            int at = before;
            int b = b0;
            for (;; ++b) {
                const int u = make_seq<C>(a, load_raw(a, b)).units_head(C::SEG) * a.Hkv;
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
        const int S = s_base[1], total = s_base[2], pos = (int)min((int64_t)blockIdx.x * S, (int64_t)total);
        walk.start(a, pos, min(total - pos, S) + pos, S, *s_b0, s_base[0]);
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
    // after a role's waits, which each lane makes for itself: its warp goes on together or not at all
    auto agree = [&] { return ok = __all_sync(kFull, ok); };
    auto wait_all = [&](uint64_t *bar, uint32_t parity) {
        ok = ok && mbar_wait(bar, parity, deadline);
        ok = __all_sync(kFull, ok);
        return ok;
    };
    Item it;
    if (w == C::W_LOAD) {
        // ---- K tile j+1, then V tile j (the order of their use); a window of
        // 32 block-table entries in registers
        const int32_t *bt = nullptr;
        int win0 = 0, went = 0, nblk = 0;
        auto tile_row = [&](const Item &i, int j, int n) {  // lanes 0..7: cache row of the tile's block
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
            return (phys * a.Hkv + i.kvh) * 16;
        };
        int kn = 0, vn = 0, cn = 0;  // tiles issued
        auto fill = [&](int kv, int row) {
            int rows[C::BPT];
#pragma unroll
            for (int i = 0; i < C::BPT; ++i) rows[i] = __shfl_sync(kFull, row, i);
            if constexpr (!C::FP8) {
                const int ns = kv ? NSV : NSK, n = kv ? vn : kn, sl = n % ns;
                if (n >= ns) wait((kv ? vempty : kempty) + sl, (n / ns - 1) & 1);
                if (!agree()) return false;
                if (kv) ++vn; else ++kn;
                uint64_t *full = (kv ? vfull : kfull) + sl;
                uint8_t *dst = (kv ? sV : sK) + sl * C::TILE;
                if (elect_one()) {
                    mbar_arrive_expect_tx(full, C::TILE);
                    const CUtensorMap *map = kv ? &tmV : &tmK;
#pragma unroll
                    for (int i = 0; i < C::BPT; ++i) tma_load_4d(dst + i * 2 * C::GROUP, map, rows[i] >> 3, full);
                }
            } else {
                const int sl = cn % NST;
                if (cn >= NST) wait(&cempty[sl], (cn / NST - 1) & 1);
                if (!agree()) return false;
                ++cn;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&cfull[sl], C::CODES);
                    const CUtensorMap *map = kv ? &tmV : &tmK;
#pragma unroll
                    for (int i = 0; i < C::BPT; ++i)
                        tma_load_2d(sC + sl * C::CODES + i * 16 * D, map, 0, rows[i], &cfull[sl]);
                }
            }
            __syncwarp();
            return true;
        };
        // the next item's first window is requested before this one's tiles
        auto first_window = [&](const Item &i) {
            return a.block_tables[(size_t)i.b * a.max_blocks + min(i.j0 * C::BPT + lane, ((i.L + 15) >> 4) - 1)];
        };
        Item nx;
        bool more = walk.next(a, nx);
        int nwent = more ? first_window(nx) : 0, n = 0, vrow = 0;
#pragma unroll 1
        while (ok && more) {
            it = nx;
            went = nwent;
            bt = a.block_tables + (size_t)it.b * a.max_blocks;
            nblk = (it.L + 15) >> 4;
            win0 = it.j0 * C::BPT;
            more = walk.next(a, nx);
            if (more) nwent = first_window(nx);
#pragma unroll 1
            for (int j = it.j0; j < it.j1 + (C::ACROSS ? 0 : 1) && ok; ++j) {
                const bool v = C::ACROSS ? n > 0 : j > it.j0;
                int row = 0;
                if (j < it.j1) {
                    row = tile_row(it, j, n++);
                    if (!fill(0, row)) break;
                }
                if (v && !fill(1, vrow)) break;
                vrow = row;
            }
        }
        if (C::ACROSS && ok && n > 0) fill(1, vrow);
        if (!ok) {  // the last copy of every slot may be in flight: wait for it, with a short fresh budget
            const uint64_t dd = drain_deadline();
            auto drain = [&](uint64_t *full, int ns, int issued) {
#pragma unroll 1
                for (int sl = 0; sl < ns; ++sl)
                    if (issued > sl) mbar_wait(&full[sl], ((issued - 1 - sl) / ns) & 1, dd);
            };
            if constexpr (!C::FP8) {
                drain(kfull, NSK, kn);
                drain(vfull, NSV, vn);
            } else {
                drain(cfull, NST, cn);
            }
            __syncwarp();
        }
    } else if (w == C::W_MMA) {
        // ---- one thread issues the MMAs (a whole warp in step, with a vote
        // after its waits, spent 1,500 clocks a step on itself)
        bool done = true;
        if (elect_one()) {
            constexpr uint32_t idS = idesc_f16kind_f32(128, KT, false, !C::FP8);
            constexpr uint32_t idO = idesc_f16kind_f32(128, D, true, !C::FP8);
            struct Ring {  // slots in turn, without divisions
                int slot;
                uint32_t phase;
                PA_DEVICE void next(int n) {
                    if (++slot == n) slot = 0, phase ^= 1;
                }
            };
            // operand descriptors of the rings' first tiles; an address is 16 bytes a unit
            const uint64_t dq = smem_desc_sw128(smem_addr(sQ), 16, 1024),
                           dk = smem_desc_sw128(smem_addr(sK), 16, C::GROUP),
                           dv = smem_desc_sw128(smem_addr(sV), 1024, C::GROUP);
            int n = 0, qc = 0;                   // steps and query tiles before this one
            Ring kr{0, 0}, vr{0, 0};             // this step's K tile; the V tile of step n - 1
            bool pfirst = false, plast = false;  // step n - 1: the first of its accumulator; the last to read its V tile
            auto scores = [&](int qslot, bool last_k, bool last_q) {  // S(n) = Q K^T
                wait(&kfull[kr.slot], kr.phase);
                // P(n-2), in S(n)'s columns, has been used
                if (n >= 2 ? !wait(&odone[n & 1], ((n >> 1) - 1) & 1) : !ok) return;
                tc_fence_after();
                const uint64_t a0 = dq + qslot * (C::TILE / 16), b0 = dk + kr.slot * (C::TILE / 16);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_mma_bf16(tmem + (n & 1) * KT, a0 + ((kk / 4) * C::ATOM + (kk % 4) * 32) / 16,
                                b0 + ((kk / 4) * 1024 + (kk % 4) * 32) / 16, idS, kk > 0);
                tc_commit(&sfull[n & 1]);
                if (last_k) tc_commit(&kempty[kr.slot]);
                if (last_q) tc_commit(&qempty[qslot]);
            };
            auto pv = [&] {  // O += P(n-1) V
                wait(&vfull[vr.slot], vr.phase);
                const int p = n - 1;
                const uint64_t b0 = dv + vr.slot * (C::TILE / 16);
                const uint32_t o0 = tmem + C::COL_O + (p & 1) * D, p0 = tmem + (p & 1) * KT;
#pragma unroll
                for (int kk = 0; kk < KT / 16; ++kk) {
                    if (kk % (KT / 32) == 0) {  // each half as its P arrives
                        if (kk > 0) tc_commit(&ohalf[p & 1]);
                        if (!wait(&pfull[(kk > 0 ? 2 : 0) + (p & 1)], (p >> 1) & 1)) return;
                        tc_fence_after();
                    }
                    tc_mma_bf16_tmem_a(o0, p0 + kk * 8, b0 + kk * 2 * C::GROUP / 16, idO, !pfirst || kk > 0);
                }
                tc_commit(&odone[p & 1]);
                if (plast) {
                    tc_commit(&vempty[vr.slot]);
                    vr.next(NSV);
                }
            };
            bool more = walk.next(a, it), was_pair = false;
#pragma unroll 1
            while (more && ok) {
                const int steps = it.steps(), pair = it.rt - 1;
#pragma unroll 1
                for (int k = 0; k < steps && ok; ++k, ++n) {
                    const int qt = pair & k, qslot = (qc + qt) & 1;
                    // the scores first, so that the tensor pipe has them while
                    // P(n-1) is computed; but P.V first where a new query tile
                    // takes the place of one that the last scores read, or a
                    // new segment's operands have not landed
                    const bool pv_first = k == 0 && (pair || was_pair || !mbar_test(&kfull[kr.slot], kr.phase) ||
                                                     !mbar_test(&qfull[qslot], (qc >> 1) & 1));
                    if (pv_first && n > 0) pv();
                    if (k <= pair) wait(&qfull[qslot], ((qc + qt) >> 1) & 1);
                    scores(qslot, !pair || qt, k >= steps - 1 - pair);
                    if (!pv_first && n > 0) pv();
                    pfirst = k < 2;
                    plast = !pair || qt;
                    if (plast) kr.next(NSK);
                }
                qc += it.rt;
                was_pair = pair;
                more = ok && walk.next(a, it);
            }
            if (ok && n > 0) pv();
            // every MMA of this CTA has completed before TMEM is released
            tc_commit(mma_done);
            done = mbar_wait(mma_done, 0, ok ? deadline : drain_deadline());
        }
        ok = __all_sync(kFull, ok && done);
    } else if (w >= C::W_QUERY && w < C::W_WIDEN) {
        // ---- query tiles, two slots in turn.  bf16: warp 10, one 3-D box per
        // 64-column atom.  E4M3: warps 10 and 11, f16(q 2^e) with e per row
        // such that its largest magnitude lies in [2^14, 2^15) (exact for
        // components within 2^-28 of it)
        int qc = 0;
#pragma unroll 1
        while (ok && (C::FP8 || w == C::W_QUERY) && walk.next(a, it)) {
            // E4M3: a negative K scale goes into the query: the softmax counts on a positive one
            const uint32_t sign = C::FP8 ? __float_as_uint(a.k_scale[it.kvh]) & 0x80000000u : 0;
#pragma unroll 1
            for (int qt = 0; qt < it.rt && ok; ++qt, ++qc) {
                const int sl = qc & 1;
                if (qc >= 2) wait(&qempty[sl], ((qc >> 1) - 1) & 1);
                if (!agree()) break;
                const int q0 = it.q0 + qt * C::QPOS;
                uint8_t *tile = sQ + sl * C::TILE;
                if constexpr (!C::FP8) {
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&qfull[sl], C::TILE);
#pragma unroll
                        for (int at = 0; at < C::NATOM; ++at)
                            tma_load_3d(tile + at * C::ATOM, &tmQ, at * 64, it.kvh * G, q0, &qfull[sl]);
                    }
                    __syncwarp();
                } else {
                    // a row is LPR lanes of 8 dims; the warp's rows RPW apart
                    constexpr int LPR = D / 8, RPW = 32 / LPR;
                    const int nrows = min(C::QPOS, it.T - it.r0 - qt * C::QPOS) * G;
                    const int ch = lane % LPR, at = ch / 8, cc = ch % 8;
#pragma unroll 1
                    for (int rb = (w - C::W_QUERY) * 64 + lane / LPR; rb < (w - C::W_QUERY + 1) * 64; rb += 8 * RPW) {
                        uint4 v[8];  // 8 rows' loads in flight
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const int r = rb + u * RPW;
                            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) +
                                                       ((size_t)(q0 + r / G) * a.Hq + (size_t)it.kvh * G + r % G) * D + ch * 8;
                            v[u] = r < nrows ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const int r = rb + u * RPW;
                            const uint32_t wd[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
                            float2 f[4];
                            float amax = 0.f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                f[e] = bf16x2_to_float2(wd[e]);
                                amax = fmax3(amax, fabsf(f[e].x), fabsf(f[e].y));
                            }
#pragma unroll
                            for (int o = LPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
                            int ex = 0;
                            if (amax > 0.f) ex = min(max(14 - ((int)((__float_as_uint(amax) >> 23) & 0xff) - 127), -100), 100);
                            const float qs = __uint_as_float(sign | (uint32_t)(127 + ex) << 23);
                            uint32_t h[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __half2 hh = __floats2half2_rn(f[e].x * qs, f[e].y * qs);
                                h[e] = *reinterpret_cast<const uint32_t *>(&hh);
                            }
                            *reinterpret_cast<uint4 *>(tile + at * C::ATOM + r * 128 + ((cc ^ (r & 7)) * 16)) =
                                make_uint4(h[0], h[1], h[2], h[3]);
                            if (ch == 0) qexp[(qc & 3) * 128 + r] = (int8_t)ex;
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&qfull[sl]);
                }
            }
        }
        if (!C::FP8 && w == C::W_QUERY) {  // the copies have landed before the CTA may exit
            const uint64_t dd = ok ? deadline : drain_deadline();
            for (int sl = 0; sl < 2; ++sl)
                if (qc > sl && !mbar_wait(&qfull[sl], ((qc - 1 - sl) >> 1) & 1, dd)) ok = false;
            __syncwarp();
        }
    } else if (w >= C::W_WIDEN) {
        if constexpr (C::FP8) {
            // ---- E4M3: thread ct widens key row ct of each staged tile into its
            // f16 operand tile
            const int ct = tid - C::W_WIDEN * 32;
            int kn = 0, vn = 0, cn = 0, n = 0;
            auto widen = [&](int kv, int kv0, int L, int nn) {
                const int ns = kv ? NSV : NSK, m = kv ? vn : kn, sl = m % ns, cs = cn % NST;
                if (!wait(&cfull[cs], (cn / NST) & 1)) return false;
                if (m >= ns && !wait((kv ? vempty : kempty) + sl, (m / ns - 1) & 1)) return false;
                if (kv) ++vn; else ++kn;
                ++cn;
                uint8_t *row = (kv ? sV : sK) + sl * C::TILE + (ct >> 3) * C::GROUP + (ct & 7) * 128;
                const uint8_t *codes = sC + cs * C::CODES + ct * D;
                const bool live = kv0 + ct < L && !((badmask[nn % C::NBAD] >> (ct >> 4)) & 1);
                uint4 src[D / 16];
#pragma unroll
                for (int u = 0; u < D / 16; ++u) {  // the codes' rows are swizzled too: conflict-free columns
                    const int ch = D == 128 ? (u ^ (ct & 7)) : (u ^ ((ct >> 1) & 3));
                    src[u] = live ? *reinterpret_cast<const uint4 *>(codes + 16 * ch) : make_uint4(0, 0, 0, 0);
                }
                uint32_t nan = 0;
#pragma unroll
                for (int u = 0; u < D / 16; ++u) {
                    const uint32_t wd[4] = {src[u].x, src[u].y, src[u].z, src[u].w};
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (e & 1) {
                            widen4_cvt(wd[e], h[2 * e], h[2 * e + 1]);
                            continue;
                        }
                        widen4(wd[e], h[2 * e], h[2 * e + 1]);
                        nan |= (wd[e] & 0x7f7f7f7fu) + 0x01010101u;  // bit 7 of a byte: its code is a NaN
                    }
                    store_chunks<C>(row, u, ct, h);
                }
                // only now, with every code used: an arrival straight behind
                // the loads let the next copy overwrite codes still on their way
                mbar_arrive(&cempty[cs]);
                if (nan & 0x80808080u) {  // a NaN has no place in the scaled range: write it
#pragma unroll 1
                    for (int d = 0; d < D; ++d) {
                        const int at = d / 64, cc = d % 64 / 8;
                        uint16_t *x = reinterpret_cast<uint16_t *>(row + at * 1024 + ((cc ^ (ct & 7)) * 16)) + d % 8;
                        if ((*x & 0x7fff) == 0x3f80) *x = 0x7fff;
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive((kv ? vfull : kfull) + sl);
                return true;
            };
            int vkv0 = 0, vL = 0;
            bool more = true;
#pragma unroll 1
            while (ok && more) {  // K tile n+1 before V tile n, as the loader; at the end the last V tile alone
                more = walk.next(a, it);
                const int cnt = more ? it.j1 - it.j0 : 1;
#pragma unroll 1
                for (int j = 0; j < cnt && ok; ++j) {
                    const int kv0 = (it.j0 + j) * KT;
#pragma unroll 1
                    for (int kv = more ? 0 : 1; kv < 2; ++kv)
                        if ((kv == 0 || n > 0) && !widen(kv, kv ? vkv0 : kv0, kv ? vL : it.L, kv ? n - 1 : n)) break;
                    vkv0 = kv0;
                    vL = it.L;
                    ++n;
                }
            }
            static_assert(C::ACROSS, "the order of this loop");
        }
    } else {
        // ---- softmax: warpgroup g takes the steps n with n % 2 == g; thread
        // = row r of the step's row tile
        const int g = w >> 2, r = (w & 3) * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)((w & 3) * 32) << 16);
        const uint32_t scol = lane_base + g * KT, ocol = lane_base + C::COL_O + g * D;
        int n = 0, kt = 0, qc = 0;
        int4 desc = make_int4(0, 0, 0, 0);
        auto make_desc = [&](const Item &i) {  // (of the share's last item)
            return make_int4(i.q0, min(2 * C::QPOS, i.T - i.r0) * G, i.kvh, walk.pieces(i));
        };
#pragma unroll 1
        while (walk.next(a, it)) {
            const int steps = it.steps(), pair = it.rt - 1;
            const int k0 = (n ^ g) & 1, qt = pair & k0;       // first step of this warpgroup, its row tile
            // one stream alone holds a row's result: each row tile of two, or
            // a single step (the other warpgroup goes on to the next item)
            const bool solo = pair || steps == 1;
            if (k0 >= steps) {
                n += steps;
                kt += it.j1 - it.j0;
                qc += it.rt;
                if (it.begins_cut()) desc = make_desc(it);
                continue;
            }
            const int nrows = min(C::QPOS, it.T - it.r0 - qt * C::QPOS) * G;
            const bool warp_live = (w & 3) * 32 < nrows, row_live = r < nrows;
            const int64_t qrow = it.q0 + qt * C::QPOS + r / G;
            const uint64_t bits = row_live ? a.mask[qrow] : 0;
            float sl2 = a.scale * kLog2e * C::OPMUL * (C::FP8 ? fabsf(a.k_scale[it.kvh]) : 1.f);
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int k = k0; k < steps; k += 2) {
                const int nn = n + k, kv0 = (it.j0 + (pair ? k >> 1 : k)) * KT;
                const bool landed = wait_all(&sfull[g], (nn >> 1) & 1);
                if (C::FP8 && landed && k == k0) {
                    sl2 *= __uint_as_float((uint32_t)(127 - qexp[((qc + qt) & 3) * 128 + r]) << 23);
                    // a K scale of zero: scores (below 2^24) that round to zero, but masked ones stay -inf
                    if (sl2 == 0.f) sl2 = 0x1p-126f;
                }
                const int t = kt + (pair ? k >> 1 : k);
                const uint32_t bad = badmask[t % C::NBAD];
                if constexpr (!C::FP8) {  // V rows past the end or of bad blocks: zero them before they meet P
                    if (kv0 + KT > it.L || bad) {
                        const bool there = wait_all(&vfull[t % NSV], (t / NSV) & 1);
                        if (there && (kv0 + r >= it.L || ((bad >> (r >> 4)) & 1))) {
                            uint8_t *vrow = sV + t % NSV * C::TILE + (r >> 3) * C::GROUP + (r & 7) * 128;
#pragma unroll
                            for (int c = 0; c < C::NATOM * 8; ++c)
                                *reinterpret_cast<uint4 *>(vrow + (c / 8) * 1024 + (c % 8) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                }
                // the keys this row may see, where the tile is not all prefix
                const bool masked = kv0 + KT > it.P || bad;
                // half a tile at a time: P.V of the first 64 keys runs while
                // the second 64 are exponentiated
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (ok && warp_live) {
                        tc_fence_after();
                        float sv[64];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float x[32];
                            tmem_ld32(scol + 64 * h + 32 * q, x);
#pragma unroll
                            for (int e = 0; e < 32; ++e) sv[32 * q + e] = x[e];
                        }
                        tmem_wait_ld();
                        if (masked) {
                            const uint64_t seen = it.T < 64 ? bits & ((1ull << it.T) - 1) : bits;
                            const int rel = kv0 + 64 * h - it.P;  // draft of the first key
                            uint64_t v = rel <= -64  ? ~0ull
                                         : rel >= 64 ? 0ull
                                         : rel < 0   ? (seen << -rel) | ((1ull << -rel) - 1)
                                                     : seen >> rel;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if ((bad >> (4 * h + i)) & 1) v &= ~(0xffffull << (16 * i));
                            const uint32_t vl = (uint32_t)v, vh = (uint32_t)(v >> 32);
#pragma unroll
                            for (int e = 0; e < 64; ++e)
                                sv[e] = (e < 32 ? vl : vh) & (1u << (e & 31)) ? sv[e] : -INFINITY;
                        }
                        float mx = -INFINITY, my = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            mx = fmax3(mx, sv[e], sv[e + 1]);
                            my = fmax3(my, sv[32 + e], sv[33 + e]);
                        }
                        const float mt = fmaxf(mx, my) * sl2;  // (the scale is positive)
                        const bool rescale = mt > m + kRescaleThreshold;
                        if (__any_sync(kFull, rescale)) {
                            const float alpha = rescale ? ex2(m - mt) : 1.f;  // m = -inf: 0
                            if (rescale) m = mt;
                            l2 = make_float2(l2.x * alpha, l2.y * alpha);
                            // O holds P.V up to the half tile before: complete
                            // for the first half (these scores were issued after it)
                            if (h > 0) wait_all(&ohalf[g], (nn >> 1) & 1);
                            if (ok && (h > 0 || k > k0)) {
                                tc_fence_after();
#pragma unroll 1
                                for (int q = 0; q < D / 16; ++q) {
                                    float o[16];
                                    tmem_ld16(ocol + 16 * q, o);
                                    tmem_wait_ld();
                                    uint32_t ou[16];
#pragma unroll
                                    for (int e = 0; e < 16; ++e) ou[e] = __float_as_uint(o[e] * alpha);
                                    tmem_st16_u(ocol + 16 * q, ou);
                                }
                            }
                        }
                        const float nb = (m == -INFINITY ? 0.f : -m) + C::PBIAS;
                        const float2 sc2 = make_float2(sl2, sl2), nb2 = make_float2(nb, nb);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 32 * q; e < 32 * q + 32; e += 2) {
                                const float2 y = ffma2(make_float2(sv[e], sv[e + 1]), sc2, nb2);
                                const float2 p = make_float2(ex2(y.x), ex2(y.y));
                                l2 = fadd2(l2, p);
                                if constexpr (C::FP8) {
                                    const __half2 hh = __floats2half2_rn(p.x, p.y);
                                    pk[e / 2 - 16 * q] = *reinterpret_cast<const uint32_t *>(&hh);
                                } else {
                                    const __nv_bfloat162 bb = __floats2bfloat162_rn(p.x, p.y);
                                    pk[e / 2 - 16 * q] = *reinterpret_cast<const uint32_t *>(&bb);
                                }
                            }
                            tmem_st16_u(scol + 32 * h + 16 * q, pk);  // over scores that this thread has read
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    mbar_arrive(&pfull[2 * h + g]);
                }
            }
            // ---- epilogue: all columns of a stream alone, or the two
            // accumulators joined, columns [g D/2, (g+1) D/2)
            const int last = n + steps - 1;  // the last step; the other stream's is last - 1
            float M = m, l = l2.x + l2.y, f0 = 1.f, f1 = 0.f;
            bool landed = true;
            if (!solo) {
                ml[g * 128 + r] = make_float2(m, l);
                named_bar_sync(kEpiBar, 256);
                const float2 ml0 = ml[r], ml1 = ml[128 + r];
                M = fmaxf(ml0.x, ml1.x);
                f0 = ml0.x == -INFINITY ? 0.f : ex2(ml0.x - M);
                f1 = ml1.x == -INFINITY ? 0.f : ex2(ml1.x - M);
                l = ml0.y * f0 + ml1.y * f1;
            }
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
                const int nn = last - u;
                if (solo && (nn & 1) != g) continue;
                landed = wait_all(&odone[nn & 1], (nn >> 1) & 1);
            }
            const float inv = (l > 0.f ? 1.f / l : l == l ? 0.f : l) * C::OPMUL * (C::FP8 ? a.v_scale[it.kvh] : 1.f);
            const uint32_t colA = lane_base + C::COL_O + (solo ? g * D : 0);
            const bool dead = l == 0.f;  // sees nothing: zeros
            const float wA = f0 * inv, wB = f1 * inv;  // (alone: f0 = 1)
            const int c0 = solo ? 0 : g * (D / 2), c1 = solo ? D : c0 + D / 2;
            const bool whole = it.whole();
            const int srow = it.slot(blockIdx.x) * 256 + qt * 128;
            auto out_row = [&](int rr) {
                return static_cast<__nv_bfloat16 *>(a.out) +
                       ((it.q0 + qt * C::QPOS + rr / G) * (int64_t)a.Hq + it.kvh * G + rr % G) * D;
            };
            if (landed && warp_live) {
                tc_fence_after();
                __nv_bfloat16 *dst = out_row(r);
                float *wo = ws.o + (size_t)(srow + r) * D;
                float zero = 0.f;  // turns NaN where an output is not finite
#pragma unroll 1
                for (int c = c0; c < c1; c += 16) {
                    float o[16];
                    tmem_ld16(colA + c, o);
                    if (solo) {  // (no second accumulator: an infinity times a weight of zero would be a NaN)
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= wA;
                    } else {
                        float ob[16];
                        tmem_ld16(colA + D + c, ob);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = fmaf(ob[e], wB, o[e] * wA);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        o[e] = dead ? 0.f : o[e];
                        zero = fmaf(o[e], 0.f, zero);
                    }
                    if (!row_live) continue;
                    if (whole) {
                        uint32_t wd[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const __nv_bfloat162 bb = __floats2bfloat162_rn(o[2 * u], o[2 * u + 1]);
                            wd[u] = *reinterpret_cast<const uint32_t *>(&bb);
                        }
                        *reinterpret_cast<uint4 *>(dst + c) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
                        *reinterpret_cast<uint4 *>(dst + c + 8) = make_uint4(wd[4], wd[5], wd[6], wd[7]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4 *>(wo + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (!whole && row_live && (solo || g == 0))
                    ws.lse[srow + r] = l > 0.f ? M + lg2(l) - C::PBIAS : l == l ? -INFINITY : l;
                // rows that an unseen draft's V spoilt
                uint32_t todo = __ballot_sync(kFull, zero != 0.f && row_live && l > 0.f && l <= 3.4028235e38f);
                const Item copy = it;  // (what a call takes by reference lives in local memory: not the loop's own)
                if (todo && it.j1 * KT > it.P && drafts_not_finite<C>(a, copy, lane)) {
#pragma unroll 1
                    while (todo) {
                        const int rl = __ffs(todo) - 1, rr = (w & 3) * 32 + rl;
                        todo &= todo - 1;
                        float acc[D / 32];
                        attend_row<C>(a, copy, qt * 128 + rr, __shfl_sync(kFull, bits, rl),
                                      __shfl_sync(kFull, M, rl) - C::PBIAS, lane, acc);
                        const float iv = __shfl_sync(kFull, inv, rl) * (1.f / C::OPMUL);
#pragma unroll
                        for (int e = 0; e < D / 32; ++e) {
                            const int d = lane * (D / 32) + e;
                            if (d < c0 || d >= c1) continue;
                            if (whole) out_row(rr)[d] = __float2bfloat16_rn(acc[e] * iv);
                            else ws.o[(size_t)(srow + rr) * D + d] = acc[e] * iv;
                        }
                    }
                }
            }
            tc_fence_before();
            if (!solo) named_bar_sync(kEpiBar, 256);  // both accumulators and (m, l) are read
            n += steps;
            kt += it.j1 - it.j0;
            qc += it.rt;
            if (it.begins_cut()) desc = make_desc(it);
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
// One warp per row.  The first pieces' sums and outputs are requested together
// with the description (their places do not depend on it, and every slot is
// there to be read), so a segment of up to kMergeAhead pieces costs one round
// trip.
constexpr int kMergeAhead = 3;

template <int D, int G>
__global__ void __launch_bounds__(128) tree_merge_kernel(const TreeArgs a, const TreeWs ws, int ctas) {
    constexpr int E = D / 32;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, g = blockIdx.x;
    auto load = [&](size_t at, float (&v)[E]) {
        const float *src = ws.o + at * D + lane * E;
        if constexpr (E == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
            const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
            v[0] = x.x, v[1] = x.y;
        }
    };
    const int4 d = __ldcg(ws.desc + g);
#pragma unroll 1
    for (int r = blockIdx.y * 4 + (threadIdx.x >> 5); r < 256; r += gridDim.y * 4) {
        auto at = [&](int p) { return (size_t)tree_piece_slot(g, p) * 256 + r; };
        float lse[kMergeAhead], o[kMergeAhead][E];
#pragma unroll
        for (int p = 0; p < kMergeAhead; ++p) {
            lse[p] = __ldcg(ws.lse + at(p));
            load(at(p), o[p]);
        }
        const int np = d.w;
        if (np < 1 || g + np > ctas || r >= d.y) return;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int p = 0; p < kMergeAhead; ++p)
            if (p < np) m = fmaxf(m, lse[p]);
        if (np > kMergeAhead) {
#pragma unroll 1
            for (int p = kMergeAhead + lane; p < np; p += 32) m = fmaxf(m, __ldcg(ws.lse + at(p)));
#pragma unroll
            for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, x));
        }
        const float mb = m == -INFINITY ? 0.f : m;
        float acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        // a piece without weight (none of its keys is visible) adds nothing
        auto add = [&](float lp, const float (&v)[E]) {
            const float wt = ex2(lp - mb);
            l += wt;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = lp == -INFINITY ? acc[e] : fmaf(wt, v[e], acc[e]);
        };
#pragma unroll
        for (int p = 0; p < kMergeAhead; ++p)
            if (p < np) add(lse[p], o[p]);
#pragma unroll 4
        for (int p = kMergeAhead; p < np; ++p) {
            float v[E];
            load(at(p), v);
            add(__ldcg(ws.lse + at(p)), v);
        }
        const float inv = l > 0.f ? 1.f / l : l == l ? 0.f : l;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) +
                             ((size_t)(d.x + r / G) * a.Hq + (size_t)d.z * G + r % G) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<__nv_bfloat162 *>(dst + e) = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
    }
}

// ---- host side
// A tensor of `rank` dims (innermost first) with byte strides for all but the
// first, copied in boxes of `box`.
bool tiled_map(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims,
               const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle) {
    auto fn = encode_fn();
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return fn && fn(map, type, rank, const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
    const cuuint64_t rows = (cuuint64_t)a.num_blocks * a.Hkv * 16;
    bool ok;
    if (C::FP8) {  // rows of D codes; a box is a block of one kv head
        const cuuint64_t dims[2] = {(cuuint64_t)C::D, rows}, strides[1] = {(cuuint64_t)C::D};
        const cuuint32_t box[2] = {(cuuint32_t)C::D, 16};
        const auto swz = C::D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
        ok = tiled_map(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.k_cache, dims, strides, box, swz) &&
             tiled_map(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.v_cache, dims, strides, box, swz);
    } else {
        const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        const auto swz = CU_TENSOR_MAP_SWIZZLE_128B;
        // 64 columns, 8 rows, column atoms, 8-row groups
        const cuuint64_t dims[4] = {64, 8, (cuuint64_t)C::NATOM, rows / 8};
        const cuuint64_t strides[3] = {(cuuint64_t)C::D * 2, 128, (cuuint64_t)C::D * 16};
        const cuuint32_t box[4] = {64, 8, (cuuint32_t)C::NATOM, 2};
        const cuuint64_t qdims[3] = {(cuuint64_t)C::D, (cuuint64_t)a.Hq, (cuuint64_t)a.total_q};
        const cuuint64_t qstrides[2] = {(cuuint64_t)C::D * 2, (cuuint64_t)a.Hq * C::D * 2};
        const cuuint32_t qbox[3] = {64, (cuuint32_t)C::G, (cuuint32_t)C::QPOS};
        ok = tiled_map(&tk, bf16, 4, a.k_cache, dims, strides, box, swz) &&
             tiled_map(&tv, bf16, 4, a.v_cache, dims, strides, box, swz) &&
             tiled_map(&tq, bf16, 3, a.q, qdims, qstrides, qbox, swz);
    }
    if (!ok) return cudaErrorInvalidValue;
    // a CTA per SM, fewer where the batch has fewer key tiles
    const long long groups = (a.max_q_len + 2 * C::QPOS - 1) / (2 * C::QPOS);
    const long long tiles_wide = (a.max_blocks + C::BPT - 1) / C::BPT;
    const int ctas = (int)std::min<long long>({(long long)a.B * a.Hkv * groups * tiles_wide, sm_count(),
                                                kMaxCtas - kMergeAhead});  // (the merge looks that far past the last)
    e = launch_pdl(tree_kernel<C>, dim3(ctas), dim3(C::NT), C::SMEM, st, a, ws, tk, tv, tq);
    if (e != cudaSuccess) return e;
    return launch_pdl(tree_merge_kernel<C::D, C::G>, dim3(ctas, 32), dim3(128), 0, st, a, ws, ctas);
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

constexpr size_t kLseBytes = 2 * kMaxCtas * 256 * sizeof(float), kDescBytes = kMaxCtas * sizeof(int4);

}  // namespace

size_t tree_ws_bytes(int D) { return kLseBytes + kDescBytes + (size_t)2 * kMaxCtas * 256 * D * sizeof(float); }

cudaError_t launch_tree(const TreeArgs &a, void *workspace, cudaStream_t st) {
    char *p = static_cast<char *>(workspace);
    const TreeWs ws{reinterpret_cast<float *>(p + kLseBytes + kDescBytes), reinterpret_cast<float *>(p),
                    reinterpret_cast<int4 *>(p + kLseBytes)};
    if (a.D == 128) return a.fp8 ? tree_by_group<128, true>(a, ws, st) : tree_by_group<128, false>(a, ws, st);
    if (a.D == 64) return a.fp8 ? tree_by_group<64, true>(a, ws, st) : tree_by_group<64, false>(a, ws, st);
    return cudaErrorNotSupported;
}

}  // namespace pa
