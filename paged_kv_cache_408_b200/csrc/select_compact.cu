// select_compact.cu -- which cached tokens to keep, and moving the kept ones
// together inside the paged cache.
//
// Select (pa_select_tokens), per (sequence, kv head) row with n cached
// tokens, a budget m, `sink` leading and `recent` trailing positions that
// always stay: if n <= m every position is kept, otherwise
//     [0, sink)  u  [n - recent, n)  u  the m - sink - recent positions of
//     [sink, n - recent) with the largest weights, ties to the lowest,
// in ascending order.  Weights are fp32, paged like the cache
// ([num_blocks][Hkv][16]); NaN counts as the largest value, -0 equals +0.
//   * The k-th largest weight is found by radix selection on order-preserving
//     32-bit keys: three histograms of 11, 11 and 10 bits, each narrowing
//     the prefix of the k-th key.  A position is then kept if its key is
//     above that key, or equals it and fewer than `need` equal keys precede
//     it, so its place in the list is
//         sink + (keys above before it) + min(equal keys before it, need):
//     one ordered count of both kinds gives every place, and the result does
//     not depend on the order in which threads or atomics run.
//   * The row is read from HBM once: its keys stay in shared memory for the
//     later passes (what does not fit is read again through L2).  Rows of
//     more than 4096 tokens are spread over a thread-block cluster: each CTA
//     keeps a contiguous part and adds its histogram to the first CTA's
//     through distributed shared memory, one word a bin and CTA (30 us for 4 x
//     65536 tokens x 8 heads, then, against 82 for every CTA reading every
//     other's histogram, 32 remote loads a thread and pass).
//   * The search ends as soon as every key with the current digits is to be
//     kept, mostly after two passes (12.7 -> 9.8 us and 30 -> 28 us).
//   * Bound: the chain of passes (latency), not bytes: 4 B a token would take
//     0.5 us for 64 sequences of U[1,2048] tokens and 8 heads (9.8 us in a
//     graph) and 1.6 us for the long rows above (28 us).
//   * The plan goes by the tables' width, since the host does not know the
//     lengths: those 64 sequences take 9.1 us in tables of 128 blocks, 21 us in
//     tables of 512 (two CTAs a row) and 152 us in tables of 8,192 (eight, most
//     of them without a token).
//     Counting the many exact zeros in registers instead of by atomics
//     changed nothing.
//
// Compact (pa_compact_kv): token keep[i] of a row moves to position
// start + i, K, V and (if given) the weights, in place.  The list ascends
// and keep[i] >= start + i, so a destination never lies above a source of
// the same or a later entry: if the entries are taken in order, in groups
// that are all read before any of the group is written, no source is
// overwritten before it was read.
//   * One cluster per (sequence, kv head); its CTAs read one group of
//     consecutive entries together into registers, meet at the cluster
//     barrier, and write.  The next group's sources lie above every
//     destination of this one, so its reads need no second barrier.
//   * The list and the block table are two dependent reads before any data
//     can be: a CTA resolves 512 entries at a time into cache rows in shared
//     memory, so that the groups' reads wait for nothing.
//   * 16-byte vectors; a thread moves the same vector of K and V.
//   * Entries that are in place already are skipped.
//   * Each moved row is read and written once.  Calls back to back, so that
//     what a kernel leaves in L2 to be written counts: 44 us for 64 x
//     U[1,2048] tokens cut to 512 (204 MB, 4.7 TB/s; one CTA a row, 384 of the
//     512 have work, and the SMs that got four of them end last), 105 us for
//     8 x 32768 E4M3 tokens halved (549 MB, 5.2 TB/s: HBM).  The kernels alone
//     take 35 and 100 us, in which a part of their writes (half of the first
//     one's) has not reached HBM; with the list read inside the group loop 72
//     and 227 us, with two CTAs an SM that request the next group before the
//     barrier 37 and 118.
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace pa {
namespace {

// ------------------------------------------------------------------ clusters
PA_DEVICE uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster: everything before is ordered before everything
// after, in every CTA of the cluster.
PA_DEVICE void cluster_sync() {
    __syncwarp();  // the aligned forms are executed by whole warps
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The two halves of cluster_sync().
PA_DEVICE void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
PA_DEVICE void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// One 32-bit word of CTA `rank`'s shared memory, at the place of `p` in this CTA's.
PA_DEVICE int dsmem_load(const int *p, uint32_t rank) {
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

PA_DEVICE int4 dsmem_load4(const int *p, uint32_t rank) {
    uint32_t a;
    int4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
PA_DEVICE void dsmem_add(const int *p, uint32_t rank, int v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Launch with a cluster of `c` CTAs along x, as a programmatic dependent.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, int c, int threads, size_t smem, cudaStream_t st,
                           Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = c;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// -------------------------------------------------------------------- select
constexpr int kSelCap = 16384;  // keys a CTA keeps in shared memory (64 KB)
constexpr int kBins = 2048;     // 11-bit digits
constexpr unsigned kFullMask = 0xffffffffu;

// Unsigned keys in the order of the weights (NaN above +inf, -0 equal to +0).
PA_DEVICE uint32_t order_key(float f) {
    if (f != f) return 0xffffffffu;
    const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int THREADS>
struct SelectSmem {
    alignas(16) int hist[3][kBins];
    int warp_a[THREADS / 32], warp_b[THREADS / 32];
    int digit, above, count;  // digit of the k-th key in this pass; keys above it; keys that have it
    int cta_a, cta_b;      // this CTA's counts, read by the cluster
};

// Sum of `v` over the threads before this one.  (The caller synchronises
// before warp_sums is used again.)
template <int THREADS>
PA_DEVICE int block_exclusive(int v, int *warp_sums, int tid) {
    const int lane = tid & 31, w = tid >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFullMask, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    // lane i sums warp i's total where warp i lies before this one
    const int s = lane < w && lane < THREADS / 32 ? warp_sums[lane] : 0;
    return __reduce_add_sync(kFullMask, s) + x - v;
}

template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
    constexpr int kSelWarps = kSelThreads / 32, BPT = kBins / kSelThreads;  // BPT: bins a thread sums
    extern __shared__ uint32_t keys[];  // keys of this CTA's part, up to kSelCap
    __shared__ SelectSmem<kSelThreads> sm;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int C = gridDim.x, rank = C > 1 ? (int)cluster_rank() : 0;
    const int h = blockIdx.y, b = blockIdx.z;
    pdl_trigger();
    for (int i = tid; i < 3 * kBins; i += kSelThreads) (&sm.hist[0][0])[i] = 0;
    pdl_wait();
    const int64_t cap = (int64_t)a.max_blocks * 16;
    int n = a.seq_lens[b];
    if (n < 0 || n > cap) {
        if (tid == 0 && rank == 0) flag_error(a.err, PA_DEVERR_BAD_LEN);
        n = 0;
    }
    const int m = min(n, a.budget);
    if (h == 0 && rank == 0 && tid == 0) a.keep_lens[b] = m;
    int32_t *keep = a.keep + ((size_t)b * a.Hkv + h) * a.budget;
    for (int i = m + rank * kSelThreads + tid; i < a.budget; i += C * kSelThreads) keep[i] = -1;
    if (n <= a.budget) {  // everything stays (uniform over the cluster)
        for (int i = rank * kSelThreads + tid; i < m; i += C * kSelThreads) keep[i] = i;
        return;
    }
    const int lo = a.sink, hi = n - a.recent;  // candidates [lo, hi): more of them than k
    const int k = a.budget - a.sink - a.recent;
    for (int i = rank * kSelThreads + tid; i < a.sink + a.recent; i += C * kSelThreads) {
        if (i < a.sink) keep[i] = i;
        else keep[a.budget - a.recent + (i - a.sink)] = hi + (i - a.sink);
    }
    if (k == 0) return;

    // ---- this CTA's part of the row: whole quads of 4 tokens, [q0, q1) quads
    const int nquad = (n + 3) >> 2, per = (nquad + C - 1) / C;
    const int q0 = min(nquad, rank * per), q1 = min(nquad, q0 + per);
    const int32_t *bt = a.block_tables + (size_t)b * a.max_blocks;
    // the keys of tokens 4q .. 4q+3; 0, which no weight has, for those that are
    // not candidates
    auto load_quad = [&](int q) {
        const int64_t blk = bt[q >> 2];
        float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (blk < 0 || blk >= a.num_blocks) flag_error(a.err, PA_DEVERR_BAD_BLOCK);
        else f = *reinterpret_cast<const float4 *>(a.weights + (blk * a.Hkv + h) * 16 + (q & 3) * 4);
        uint4 u = make_uint4(order_key(f.x), order_key(f.y), order_key(f.z), order_key(f.w));
        const int t = 4 * q;
        if (t < lo || t + 4 > hi) {
            if (t < lo || t >= hi) u.x = 0;
            if (t + 1 < lo || t + 1 >= hi) u.y = 0;
            if (t + 2 < lo || t + 2 >= hi) u.z = 0;
            if (t + 3 < lo || t + 3 >= hi) u.w = 0;
        }
        return u;
    };
    auto quad = [&](int q) {  // the same, from shared memory where it is kept
        const int i = q - q0;
        return i < kSelCap / 4 ? reinterpret_cast<const uint4 *>(keys)[i] : load_quad(q);
    };
    if (C > 1) cluster_arrive();  // (waited for before the first remote add: that CTA has zeroed its bins, too)
    __syncthreads();              // the histograms are zero
    for (int q = q0 + tid; q < q1; q += kSelThreads) {
        const uint4 u = load_quad(q);
        if (q - q0 < kSelCap / 4) reinterpret_cast<uint4 *>(keys)[q - q0] = u;
        const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (e[x]) atomicAdd(&sm.hist[0][e[x] >> 21], 1);
    }

    // ---- the k-th largest key, 11, 11 and 10 bits at a time; or, as soon as
    // every key with the current prefix is to be taken, the one below them
    uint32_t prefix = 0;
    int need = k;  // keys still to take among those with the current prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        if (pass > 0) {
            const int above_shift = pass == 1 ? 21 : 10, mask = pass == 1 ? kBins - 1 : 1023;
            for (int q = q0 + tid; q < q1; q += kSelThreads) {
                const uint4 u = quad(q);
                const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (e[x] && (e[x] >> above_shift) == (prefix >> above_shift))
                        atomicAdd(&sm.hist[pass][(e[x] >> shift) & mask], 1);
            }
        }
        __syncthreads();
        if (C > 1) {  // add this CTA's bins to the first CTA's
            if (pass == 0) cluster_wait();
            if (rank > 0)
                for (int i = tid; i < kBins; i += kSelThreads)
                    if (sm.hist[pass][i]) dsmem_add(&sm.hist[pass][i], 0, sm.hist[pass][i]);
            cluster_sync();
        }
        // thread t sums the bins of BPT digits, highest digits first
        int bin[BPT], sum = 0;
        const int d0 = kBins - BPT * (tid + 1);  // its lowest digit
#pragma unroll
        for (int x = 0; x < BPT; x += 4) {
            const int4 v = C > 1 ? dsmem_load4(&sm.hist[pass][d0 + x], 0) : *reinterpret_cast<const int4 *>(&sm.hist[pass][d0 + x]);
            bin[x] = v.x, bin[x + 1] = v.y, bin[x + 2] = v.z, bin[x + 3] = v.w;
            sum += v.x + v.y + v.z + v.w;
        }
        int above = block_exclusive<kSelThreads>(sum, sm.warp_a, tid);  // keys with a higher digit
#pragma unroll
        for (int x = BPT - 1; x >= 0; --x) {
            if (above < need && above + bin[x] >= need) {
                sm.digit = d0 + x;
                sm.above = above;
                sm.count = bin[x];
            }
            above += bin[x];
        }
        __syncthreads();
        prefix |= (uint32_t)sm.digit << shift;
        need -= sm.above;
        if (need == sm.count) {  // (uniform over the cluster)
            --prefix;
            need = 0;
            break;
        }
        __syncthreads();
    }
    __syncthreads();

    // ---- the places: warp w counts its contiguous part of the CTA's quads,
    // then walks it again with the counts of everything before it
    const uint32_t kth = prefix;
    const int cnt = q1 - q0, wper = (cnt + kSelWarps - 1) / kSelWarps;
    const int wq0 = min(q1, q0 + w * wper), wq1 = min(q1, wq0 + wper);
    int gt = 0, eq = 0;
    for (int q = wq0 + lane; q < wq1; q += 32) {
        const uint4 u = quad(q);
        const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            gt += e[x] > kth;
            eq += e[x] == kth;  // (kth is a weight's key or, with need 0, whatever is below one)
        }
    }
    gt = __reduce_add_sync(kFullMask, gt);
    eq = __reduce_add_sync(kFullMask, eq);
    if (lane == 0) {
        sm.warp_a[w] = gt;
        sm.warp_b[w] = eq;
    }
    __syncthreads();
    int gbefore = 0, ebefore = 0, gall = 0, eall = 0;
#pragma unroll
    for (int i = 0; i < kSelWarps; ++i) {
        const int ga = sm.warp_a[i], ea = sm.warp_b[i];
        gbefore += i < w ? ga : 0;
        ebefore += i < w ? ea : 0;
        gall += ga;
        eall += ea;
    }
    if (C > 1) {
        if (tid == 0) {
            sm.cta_a = gall;
            sm.cta_b = eall;
        }
        cluster_sync();
        const int ga = lane < rank ? dsmem_load(&sm.cta_a, lane) : 0, ea = lane < rank ? dsmem_load(&sm.cta_b, lane) : 0;
        gbefore += __reduce_add_sync(kFullMask, ga);
        ebefore += __reduce_add_sync(kFullMask, ea);
    }
    for (int qb = wq0; qb < wq1; qb += 32) {
        const int q = qb + lane;
        uint32_t e[4] = {0, 0, 0, 0};
        if (q < wq1) {
            const uint4 u = quad(q);
            e[0] = u.x, e[1] = u.y, e[2] = u.z, e[3] = u.w;
        }
        int g = 0, t = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            g += e[x] > kth;
            t += e[x] == kth;
        }
        // both counts of a lane are at most 4: scan them packed
        int pk = g | (t << 16);
        const int mine = pk;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFullMask, pk, o);
            if (lane >= o) pk += y;
        }
        const int all = __shfl_sync(kFullMask, pk, 31), ex = pk - mine;
        int gb = gbefore + (ex & 0xffff), eb = ebefore + (ex >> 16);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const bool isg = e[x] > kth, ise = e[x] == kth;
            if (isg || (ise && eb < need)) keep[a.sink + gb + min(eb, need)] = 4 * q + x;
            gb += isg;
            eb += ise;
        }
        gbefore += all & 0xffff;
        ebefore += all >> 16;
    }
    if (C > 1) cluster_sync();  // no CTA leaves while its counts may still be read
}

// ------------------------------------------------------------------- compact
constexpr int kCmpThreads = 256;
constexpr int kCmpCtas = 4;     // CTAs an SM: one's reads run during another's barrier and writes
constexpr int kCmpVec = 4;      // K (and V) vectors a thread moves per group
constexpr int kCmpList = 512;   // entries a CTA resolves at a time

template <int VPR>  // 16-byte vectors per token row
__global__ void __launch_bounds__(kCmpThreads, kCmpCtas) compact_kernel(const CompactArgs a) {
    // TOK: entries a vector index u covers; GRP: entries a CTA reads per group
    constexpr int U = kCmpVec, TOK = kCmpThreads / VPR, GRP = U * TOK, NG = kCmpList / GRP;
    __shared__ int64_t s_src[2][kCmpList], s_dst[2][kCmpList];  // cache rows; dst -1: nothing to move
    const int tid = threadIdx.x, vec = tid % VPR, tsub = tid / VPR;
    const int C = gridDim.x, rank = C > 1 ? (int)cluster_rank() : 0;
    const int h = blockIdx.y, b = blockIdx.z;
    pdl_trigger();
    pdl_wait();
    const int64_t cap = (int64_t)a.max_blocks * 16;
    const int n = a.keep_lens[b];
    const int64_t start = a.start ? a.start[b] : 0;
    if (n < 0 || n > a.max_keep || start < 0 || start + n > cap) {  // uniform over the cluster
        if (tid == 0 && rank == 0) flag_error(a.err, PA_DEVERR_BAD_LEN);
        return;
    }
    const int32_t *keep = a.keep + ((size_t)b * a.keep_heads + (a.keep_heads > 1 ? h : 0)) * a.max_keep;
    const int32_t *bt = a.block_tables + (size_t)b * a.max_blocks;
    uint4 *kc = static_cast<uint4 *>(a.k_cache), *vc = static_cast<uint4 *>(a.v_cache);

    // this CTA's groups are g C + rank, GRP entries each; group g's rows in
    // buffer (g / NG) % 2
    auto resolve = [&](int g0) {  // groups g0 .. g0 + NG - 1
#pragma unroll
        for (int e = tid; e < kCmpList; e += kCmpThreads) {
            const int64_t i = ((int64_t)(g0 + e / GRP) * C + rank) * GRP + e % GRP;
            int64_t src = -1, dst = -1;
            if (i < n) {
                const int64_t p = keep[i], to = start + i, prev = i > 0 ? keep[i - 1] : -1;
                if (p < to || p >= cap || prev >= p) {
                    flag_error(a.err, PA_DEVERR_BAD_PAIR);
                } else if (p != to) {
                    const int64_t sb = bt[p >> 4], db = bt[to >> 4];
                    if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) {
                        flag_error(a.err, PA_DEVERR_BAD_BLOCK);
                    } else {
                        src = (sb * a.Hkv + h) * 16 + (p & 15);
                        dst = (db * a.Hkv + h) * 16 + (to & 15);
                    }
                }
            }
            s_src[g0 / NG & 1][e] = src;
            s_dst[g0 / NG & 1][e] = dst;
        }
        __syncthreads();
    };
    struct Group {
        uint4 k[U], v[U];
        float wt[U];
        int64_t dst[U];
    };
    auto load = [&](int g, Group &x) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = g % NG * GRP + u * TOK + tsub;
            const int64_t src = s_src[g / NG & 1][e];
            x.dst[u] = s_dst[g / NG & 1][e];
            if (x.dst[u] >= 0) {
                x.k[u] = kc[src * VPR + vec];
                x.v[u] = vc[src * VPR + vec];
                if (a.weights && vec == 0) x.wt[u] = a.weights[src];
            }
        }
    };
    auto store = [&](const Group &x) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (x.dst[u] >= 0) {
                kc[x.dst[u] * VPR + vec] = x.k[u];
                vc[x.dst[u] * VPR + vec] = x.v[u];
                if (a.weights && vec == 0) a.weights[x.dst[u]] = x.wt[u];
            }
    };
    const int groups = (int)(((int64_t)n + (int64_t)C * GRP - 1) / ((int64_t)C * GRP));  // the same in every CTA of the cluster
    if (groups == 0) return;
    for (int g = 0; g < groups; ++g) {
        if (g % NG == 0) resolve(g);
        Group x;
        load(g, x);
        if (C > 1) cluster_sync();
        else __syncthreads();
        store(x);
    }
}

template <int VPR>
cudaError_t run_compact(const CompactArgs &a, cudaStream_t st) {
    // CTAs a row: as many as its entries fill, while the grid stays within one
    // wave
    const int group = kCmpVec * kCmpThreads / VPR;  // entries one CTA reads per group
    const long long rows = (long long)a.B * a.Hkv;
    int c = 1;
    while (c < 8 && 2 * rows * c <= (long long)kCmpCtas * sm_count() && (long long)c * group < a.max_keep) c *= 2;
    return launch_cluster(compact_kernel<VPR>, dim3(c, a.Hkv, a.B), c, kCmpThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_select(const SelectArgs &a, cudaStream_t st) {
    // rows of up to 4096 tokens: one CTA of 256 threads each (half the warps
    // of 512, whose scans cost more than the tokens); longer ones: a cluster
    // of CTAs of 512 threads, 4096 tokens each as far as 8 CTAs go
    const int64_t cap = (int64_t)a.max_blocks * 16;
    if (cap <= 4096)
        return launch_cluster(select_kernel<256>, dim3(1, a.Hkv, a.B), 1, 256, (size_t)cap * 4, st, a);
    static std::mutex mu;
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            e = cudaFuncSetAttribute(select_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCap * 4);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    int c = 2;
    while (c < 8 && cap > (int64_t)c * 4096) c *= 2;
    const int64_t part = std::min<int64_t>(kSelCap, (cap + c - 1) / c + 4);
    return launch_cluster(select_kernel<512>, dim3(c, a.Hkv, a.B), c, 512, (size_t)((part + 3) / 4) * 16, st, a);
}

cudaError_t launch_compact(const CompactArgs &a, cudaStream_t st) {
    switch (a.D * a.elem_bytes / 16) {
        case 4: return run_compact<4>(a, st);
        case 8: return run_compact<8>(a, st);
        case 16: return run_compact<16>(a, st);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace pa
