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
//     later passes (what does not fit is read again through L2).  Long rows
//     are spread over a thread-block cluster: each CTA keeps a contiguous
//     part, the histograms and the counts are added over distributed shared
//     memory.
//   * Bound: the chain of passes (latency), not bytes: 4 B per token.
//
// Compact (pa_compact_kv): token keep[i] of a row moves to position
// start + i, K, V and (if given) the weights, in place.  The list ascends
// and keep[i] >= start + i, so a destination never lies above a source of
// the same or a later entry: if the entries are taken in order, in groups
// that are all read before any of the group is written, no source is
// overwritten before it was read.
//   * One cluster per (sequence, kv head); its CTAs read one group of
//     consecutive entries together into registers, meet at the cluster
//     barrier, and write.  The next group is read before the barrier: its
//     sources lie above every destination of the current group.
//   * 16-byte vectors; a thread moves the same vector of K and V, so the
//     list and the block table are looked up once for both.
//   * Entries that are in place already are skipped.
//   * Bound: HBM, each moved row read and written once.
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
// One 32-bit word of CTA `rank`'s shared memory, at the place of `p` in this CTA's.
PA_DEVICE int dsmem_load(const int *p, uint32_t rank) {
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
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
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelCap = 16384;  // keys a CTA keeps in shared memory (64 KB)
constexpr int kBins = 2048;     // 11-bit digits
constexpr unsigned kFullMask = 0xffffffffu;

// Unsigned keys in the order of the weights (NaN above +inf, -0 equal to +0).
PA_DEVICE uint32_t order_key(float f) {
    if (f != f) return 0xffffffffu;
    const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct SelectSmem {
    int hist[3][kBins];
    int warp_a[kSelWarps], warp_b[kSelWarps];
    int digit, above;      // digit of the k-th key in this pass; keys above it
    int cta_a, cta_b;      // this CTA's counts, read by the cluster
};

// Sum of `v` over the threads before this one (exclusive), and over all.
PA_DEVICE int block_exclusive(int v, int *warp_sums, int tid, int *total) {
    const int lane = tid & 31, w = tid >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFullMask, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kSelWarps; ++i) {
        const int s = warp_sums[i];
        before += i < w ? s : 0;
        all += s;
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
    extern __shared__ uint32_t keys[];  // [kSelCap] keys of this CTA's part
    __shared__ SelectSmem sm;
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
    auto load_quad = [&](int q) {  // the keys of tokens 4q .. 4q+3
        const int64_t blk = bt[q >> 2];
        float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (blk < 0 || blk >= a.num_blocks) flag_error(a.err, PA_DEVERR_BAD_BLOCK);
        else f = *reinterpret_cast<const float4 *>(a.weights + (blk * a.Hkv + h) * 16 + (q & 3) * 4);
        return make_uint4(order_key(f.x), order_key(f.y), order_key(f.z), order_key(f.w));
    };
    auto quad = [&](int q) {  // the same, from shared memory where it is kept
        const int i = q - q0;
        return i < kSelCap / 4 ? reinterpret_cast<const uint4 *>(keys)[i] : load_quad(q);
    };
    __syncthreads();  // the histograms are zero
    for (int q = q0 + tid; q < q1; q += kSelThreads) {
        const uint4 u = load_quad(q);
        if (q - q0 < kSelCap / 4) reinterpret_cast<uint4 *>(keys)[q - q0] = u;
        const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (4 * q + x >= lo && 4 * q + x < hi) atomicAdd(&sm.hist[0][e[x] >> 21], 1);
    }

    // ---- the k-th largest key, 11, 11 and 10 bits at a time
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
                    if ((e[x] >> above_shift) == (prefix >> above_shift) && 4 * q + x >= lo && 4 * q + x < hi)
                        atomicAdd(&sm.hist[pass][(e[x] >> shift) & mask], 1);
            }
        }
        if (C > 1) cluster_sync();
        else __syncthreads();
        // thread t sums the cluster's bins of 4 digits, highest digits first
        int bin[4], sum = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int d = kBins - 1 - (4 * tid + x);
            bin[x] = 0;
            if (C > 1) {
                for (int r = 0; r < C; ++r) bin[x] += dsmem_load(&sm.hist[pass][d], r);
            } else {
                bin[x] = sm.hist[pass][d];
            }
            sum += bin[x];
        }
        int total;
        int above = block_exclusive(sum, sm.warp_a, tid, &total);  // keys with a higher digit
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (above < need && above + bin[x] >= need) {
                sm.digit = kBins - 1 - (4 * tid + x);
                sm.above = above;
            }
            above += bin[x];
        }
        __syncthreads();
        prefix |= (uint32_t)sm.digit << shift;
        need -= sm.above;
        __syncthreads();
    }

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
            const bool in = 4 * q + x >= lo && 4 * q + x < hi;
            gt += in && e[x] > kth;
            eq += in && e[x] == kth;
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
        for (int r = 0; r < rank; ++r) {
            gbefore += dsmem_load(&sm.cta_a, r);
            ebefore += dsmem_load(&sm.cta_b, r);
        }
    }
    for (int qb = wq0; qb < wq1; qb += 32) {
        const int q = qb + lane;
        uint32_t e[4] = {0, 0, 0, 0};
        bool in[4];
        if (q < wq1) {
            const uint4 u = quad(q);
            e[0] = u.x, e[1] = u.y, e[2] = u.z, e[3] = u.w;
        }
        int g = 0, t = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            in[x] = q < wq1 && 4 * q + x >= lo && 4 * q + x < hi;
            g += in[x] && e[x] > kth;
            t += in[x] && e[x] == kth;
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
            if (!in[x]) continue;
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
constexpr int kCmpVec = 4;  // K (and V) vectors a thread moves per group

template <int VPR>  // 16-byte vectors per token row
__global__ void __launch_bounds__(kCmpThreads) compact_kernel(const CompactArgs a) {
    constexpr int U = kCmpVec, TOK = kCmpThreads / VPR;  // tokens per vector index u
    const int tid = threadIdx.x, vec = tid % VPR, tsub = tid / VPR;
    const int C = gridDim.x, rank = C > 1 ? (int)cluster_rank() : 0;
    const int h = blockIdx.y, b = blockIdx.z;
    pdl_trigger();
    pdl_wait();
    const int64_t cap = (int64_t)a.max_blocks * 16;
    int n = a.keep_lens[b];
    const int64_t start = a.start ? a.start[b] : 0;
    if (n < 0 || n > a.max_keep || start < 0 || start + n > cap) {  // uniform over the cluster
        if (tid == 0 && rank == 0) flag_error(a.err, PA_DEVERR_BAD_LEN);
        return;
    }
    const int32_t *keep = a.keep + ((size_t)b * a.keep_heads + (a.keep_heads > 1 ? h : 0)) * a.max_keep;
    const int32_t *bt = a.block_tables + (size_t)b * a.max_blocks;
    uint4 *kc = static_cast<uint4 *>(a.k_cache), *vc = static_cast<uint4 *>(a.v_cache);

    struct Group {
        uint4 k[U], v[U];
        float wt[U];
        int64_t dst[U];  // destination row, or -1: nothing to move
    };
    auto row_of = [&](int64_t pos) -> int64_t {  // cache row of a position, or -1
        const int64_t blk = bt[pos >> 4];
        if (blk < 0 || blk >= a.num_blocks) {
            flag_error(a.err, PA_DEVERR_BAD_BLOCK);
            return -1;
        }
        return (blk * a.Hkv + h) * 16 + (pos & 15);
    };
    // entries [i0, i0 + U * TOK) of the list, read into registers
    auto load = [&](int64_t i0, Group &g) {
        int64_t src[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * TOK + tsub;
            src[u] = -1;
            g.dst[u] = -1;
            if (i < n) {
                const int64_t p = keep[i], to = start + i;
                if (p < to || p >= cap || (i > 0 && keep[i - 1] >= p)) {
                    flag_error(a.err, PA_DEVERR_BAD_PAIR);
                } else if (p != to) {
                    src[u] = row_of(p);
                    g.dst[u] = src[u] < 0 ? -1 : row_of(to);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (g.dst[u] >= 0) {
                g.k[u] = kc[src[u] * VPR + vec];
                g.v[u] = vc[src[u] * VPR + vec];
                if (a.weights && vec == 0) g.wt[u] = a.weights[src[u]];
            }
    };
    auto store = [&](const Group &g) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (g.dst[u] >= 0) {
                kc[g.dst[u] * VPR + vec] = g.k[u];
                vc[g.dst[u] * VPR + vec] = g.v[u];
                if (a.weights && vec == 0) a.weights[g.dst[u]] = g.wt[u];
            }
    };
    const int64_t step = (int64_t)C * U * TOK;
    Group cur, nxt;
    int64_t i0 = (int64_t)rank * U * TOK;
    load(i0, cur);
    for (int64_t base = 0; base < n; base += step) {  // the same trips in every CTA of the cluster
        i0 += step;
        load(i0, nxt);
        if (C > 1) cluster_sync();
        else __syncthreads();
        store(cur);
        cur = nxt;
    }
}

template <int VPR>
cudaError_t run_compact(const CompactArgs &a, cudaStream_t st) {
    const int group = kCmpVec * kCmpThreads / VPR;  // entries one CTA reads per group
    const long long rows = (long long)a.B * a.Hkv;
    int c = 1;
    while (c < 8 && rows * c < 4LL * sm_count() && (long long)c * group < a.max_keep) c *= 2;
    return launch_cluster(compact_kernel<VPR>, dim3(c, a.Hkv, a.B), c, kCmpThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_select(const SelectArgs &a, cudaStream_t st) {
    static std::mutex mu;
    static bool ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCap * 4);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    // the longest row a CTA takes alone: 4096 tokens
    const int64_t cap = (int64_t)a.max_blocks * 16;
    int c = 1;
    while (c < 8 && cap > (int64_t)c * 4096) c *= 2;
    const int64_t part = std::min<int64_t>(kSelCap, (cap + c - 1) / c + 4);
    return launch_cluster(select_kernel, dim3(c, a.Hkv, a.B), c, kSelThreads, (size_t)((part + 3) / 4) * 16, st, a);
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
