// weights.cu -- a decode step that also adds every cached token's attention
// weight to a running sum kept beside the cache.
//
// out as in pa_decode; for token t of sequence b, kv head k:
//     w[slot(b, t)][k] = (t < seen[b] ? w : 0) + sum_{h in group k} p_h(t),
//     p_h(t) = 2^(s_h(t) - L_h),  s = scale log2(e) q_h . k_t,
//     L_h the log2-sum-exp of s_h over the sequence.
//
// A weight needs its row's whole sum, so it takes a second pass over the
// scores.  The decode kernel (its balanced split and streaming unchanged)
// leaves them in the workspace in fp32, 4 B a token and query head against
// 2 D bytes a token and kv head (E4M3; 4 D for bf16) of K and V: reading K
// again instead would cost D (2 D) bytes a token and kv head.  fp32, because
// the sums that selection compares are fp32: a score rounded to f16 would
// move a weight by up to |s| 2^-11.
// K and V are read with the evict-first policy, so that the scores are still
// in L2 when they are read back (E4M3 below: 143 -> 139 us).
// The finishing kernel, a programmatic dependent, has for each (sequence, kv
// head) CTAs that merge the pieces' outputs and, to add the weights, CTAs
// that take a share of the tokens: the pieces' log2-sum-exps give L_h, and
// each thread updates 4 tokens at a time (16 B of sums, 16 G B of scores,
// loaded before L_h is known).
//
// Bound: HBM.  64 sequences of U[1,2048] tokens, 8 kv heads of 4 x 128: 61 us
// for 275 MB (57 us attending at 4.8 TB/s, as pa_decode does); E4M3, 8 x
// 32768 tokens, groups of 8: 140 us for 554 MB (126 us attending: the
// tensor-core path issues ~500 instructions a block and warp).  One sequence
// of 700 tokens: 12.5 us in a graph, latency; shares down to 2 cost units over all SMs
// took the attending from 42 us (pa_decode's smallest share is 16) to 12.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace pa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTokens = 4 * kThreads;  // tokens a CTA updates per step

// log2-sum-exp over the pieces of one row, by one warp: the pieces' values
// at lse[slot(p) * G].
PA_DEVICE int piece_slot(int first, int p) { return (first + p) * 2 + (p == 0 ? 1 : 0); }

template <int G>
PA_DEVICE float row_lse(const float *lse, int first, int np, int lane) {
    float m = -INFINITY, l = 0.f;
    for (int p = lane; p < np; p += 32) m = fmaxf(m, __ldcg(lse + (size_t)piece_slot(first, p) * G));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float mb = m == -INFINITY ? 0.f : m;
    for (int p = lane; p < np; p += 32) l += ex2(__ldcg(lse + (size_t)piece_slot(first, p) * G) - mb);
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    return l > 0.f ? mb + lg2(l) : l == l ? INFINITY : l;  // no weight at all: 2^-inf = 0 for every token
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads) finish_kernel(const DecodeArgs a, float *__restrict__ weights,
                                                          const int32_t *__restrict__ seen, int mc) {
    constexpr int E = D / 32;
    __shared__ float s_lse[G];
    __shared__ float s_acc[kWarps][D];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int kvh = blockIdx.y, b = blockIdx.z;
    pdl_trigger();
    pdl_wait();
    const size_t seg = (size_t)b * a.Hkv + kvh, row0 = (size_t)b * a.Hq + (size_t)kvh * G;
    const int len = a.seq_lens[b];
    const int np = __ldcg(a.ws_np + seg);
    if (len <= 0 || len > a.max_blocks * 16) return;  // the decode kernel wrote the rows (and flagged a bad length)
    const int first = np > 1 ? __ldcg(a.ws_first + seg) : 0;
    const bool ok = np >= 1 && first >= 0 && first + np <= kMaxScoreWarps;  // else the decode kernel gave up (flagged)

    if ((int)blockIdx.x < mc) {  // ---- merge the pieces of G / mc heads: sum_p 2^(lse_p - L) o_p
        if (np == 1 || !ok) return;  // the decode kernel wrote the rows
        const int heads = G / mc, per = kWarps / heads;  // `per` warps a head, each every per-th piece
        const int h = blockIdx.x * heads + w / per;
        const float *lse = a.ws_lse + h, *op = a.ws_o + (size_t)h * D + lane * E;
        const float L = row_lse<G>(lse, first, np, lane);
        float acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
        for (int p = w % per; p < np; p += per) {
            const size_t at = (size_t)piece_slot(first, p) * G;
            const float wt = ex2(__ldcg(lse + at) - L);
            float v[E];
            if constexpr (E == 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(op + at * D));
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
            } else {
                const float2 x = __ldcg(reinterpret_cast<const float2 *>(op + at * D));
                v[0] = x.x, v[1] = x.y;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, v[e], acc[e]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) s_acc[w][lane * E + e] = acc[e];
        __syncthreads();
        for (int i = tid; i < heads * D / 2; i += kThreads) {
            const int hh = i / (D / 2), d = i % (D / 2) * 2;
            float x = 0.f, y = 0.f;
            for (int k = hh * per; k < (hh + 1) * per; ++k) x += s_acc[k][d], y += s_acc[k][d + 1];
            reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                               (row0 + blockIdx.x * heads + hh) * D)[d / 2] = __floats2bfloat162_rn(x, y);
        }
        return;
    }

    // ---- add the weights
    const int t0 = (((int)blockIdx.x - mc) * kThreads + tid) * 4, step = ((int)gridDim.x - mc) * kTokens;
    if (t0 - tid * 4 >= len) return;  // (uniform)
    const float *sc = a.scores + seg * a.max_blocks * 16 * G;
    const int32_t *bt = a.block_tables + (size_t)b * a.max_blocks;
    const int old = seen ? seen[b] : len;
    float s[G][4], x[4];
    float *slot = nullptr;
    auto load = [&](int t) {
        const int64_t blk = bt[t >> 4];
        slot = nullptr;
        if (blk < 0 || blk >= a.num_blocks) return;  // flagged by the decode kernel
        slot = weights + (blk * a.Hkv + kvh) * 16 + (t & 15);
        const float *src = sc + (size_t)(t >> 4) * 16 * G + (t & 15);
#pragma unroll
        for (int h = 0; h < G; ++h) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + h * 16));
            s[h][0] = v.x, s[h][1] = v.y, s[h][2] = v.z, s[h][3] = v.w;
        }
        const float4 v = *reinterpret_cast<const float4 *>(slot);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    };
    if (t0 < len) load(t0);  // the first step's loads do not wait for the sums
    if (!ok) return;
    for (int h = w; h < G; h += kWarps) {
        const float L = np > 1 ? row_lse<G>(a.ws_lse + h, first, np, lane) : __ldcg(a.ws_row_lse + row0 + h);
        if (lane == 0) s_lse[h] = L == -INFINITY ? INFINITY : L;
    }
    __syncthreads();
    float L[G];
#pragma unroll
    for (int h = 0; h < G; ++h) L[h] = s_lse[h];
    for (int t = t0; t < len; t += step) {
        if (t > t0) load(t);
        if (!slot) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float sum = 0.f;
#pragma unroll
            for (int h = 0; h < G; ++h) sum += ex2(s[h][i] - L[h]);
            x[i] = (t + i < old ? x[i] : 0.f) + sum;
        }
        if (t + 4 <= len) {
            *reinterpret_cast<float4 *>(slot) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (t + i < len) slot[i] = x[i];
        }
    }
}

template <int D, int G>
cudaError_t finish(const DecodeArgs &a, float *weights, const int32_t *seen, cudaStream_t st) {
    // CTAs per (sequence, kv head): with few of them each is cut into many
    // pieces, so a CTA merges one head; with many, one merges all heads.
    // Token shares: as many as the tokens fill, within one wave of the grid.
    const long long rows = (long long)a.B * a.Hkv, wave = 2048 / kThreads * (long long)sm_count();
    const int mc = rows < sm_count() ? G : 1;
    const long long cx = std::min<long long>(std::max<long long>(1, wave / rows - mc),
                                             ((long long)a.max_blocks * 16 + kTokens - 1) / kTokens);
    return launch_pdl(finish_kernel<D, G>, dim3((unsigned)(cx + mc), a.Hkv, a.B), dim3(kThreads), 0, st, a, weights, seen,
                      mc);
}

template <int D>
cudaError_t finish_by_group(const DecodeArgs &a, float *weights, const int32_t *seen, cudaStream_t st) {
    switch (a.Hq / a.Hkv) {
        case 1: return finish<D, 1>(a, weights, seen, st);
        case 2: return finish<D, 2>(a, weights, seen, st);
        case 4: return finish<D, 4>(a, weights, seen, st);
        case 8: return finish<D, 8>(a, weights, seen, st);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace

namespace {

// The workspace: piece counts, first warps, log2-sum-exps of whole rows,
// pieces, scores; every region 256-byte aligned.
struct Layout {
    size_t np, first, row, o, lse, scores, total;
};

Layout layout(int B, int Hq, int Hkv, int D, int max_blocks) {
    auto round256 = [](size_t n) { return (n + 255) & ~(size_t)255; };
    const size_t slots = 2 * (size_t)kMaxScoreWarps * (Hq / Hkv);
    Layout l{};
    l.first = l.np + round256((size_t)B * Hkv * 4);
    l.row = l.first + round256((size_t)B * Hkv * 4);
    l.o = l.row + round256((size_t)B * Hq * 4);
    l.lse = l.o + slots * D * 4;
    l.scores = l.lse + round256(slots * 4);
    l.total = l.scores + (size_t)B * Hq * max_blocks * 16 * 4;
    return l;
}

}  // namespace

size_t weights_ws_bytes(int B, int Hq, int Hkv, int D, int max_blocks) { return layout(B, Hq, Hkv, D, max_blocks).total; }

cudaError_t launch_decode_weights(const DecodeArgs &d, float *weights, const int32_t *seen, void *workspace,
                                  cudaStream_t st) {
    DecodeArgs a = d;
    const Layout l = layout(a.B, a.Hq, a.Hkv, a.D, a.max_blocks);
    char *ws = static_cast<char *>(workspace);
    a.partition_tokens = 0;
    a.ws_np = reinterpret_cast<int *>(ws + l.np);
    a.ws_first = reinterpret_cast<int *>(ws + l.first);
    a.ws_row_lse = reinterpret_cast<float *>(ws + l.row);
    a.ws_o = reinterpret_cast<float *>(ws + l.o);
    a.ws_lse = reinterpret_cast<float *>(ws + l.lse);
    a.scores = reinterpret_cast<float *>(ws + l.scores);
    const cudaError_t e = launch_decode_scores(a, st);
    if (e != cudaSuccess) return e;
    return a.D == 128 ? finish_by_group<128>(a, weights, seen, st) : finish_by_group<64>(a, weights, seen, st);
}

}  // namespace pa
