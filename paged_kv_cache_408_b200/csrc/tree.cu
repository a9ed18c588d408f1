// tree.cu -- attention of drafted tokens over a paged prefix and over the
// drafts each one may see (verification of a token tree).
//
// Row i of sequence b (rows cu_q[b] .. cu_q[b+1]-1, at most 64) attends, per
// query head, to keys [0, P_b) and to key P_b + j for every j with bit j of
// mask[row] set:
//     out = sum_t softmax_t(scale q . k_t) v_t    over those keys,
// zero where there are none.
//
// One warp per (row, query head): lane l holds D/32 dims, walks the keys
// with an online softmax.
#include "common.cuh"
#include "kernels.h"

namespace pa {
namespace {

template <int D, bool FP8>
__global__ void __launch_bounds__(128) tree_kernel(const TreeArgs a) {
    constexpr int E = D / 32;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long u = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int row = (int)(u / a.Hq), h = (int)(u % a.Hq);
    if (row >= a.total_q) return;
    const int kvh = h / (a.Hq / a.Hkv);
    int lo = 0, hi = a.B;  // the last b with cu_q[b] <= row
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_q[mid] <= row) lo = mid; else hi = mid;
    }
    const int b = lo, T = a.cu_q[b + 1] - a.cu_q[b], P = a.prefix_lens[b];
    if (row < a.cu_q[b] || row >= a.cu_q[b + 1]) return;
    if (T > a.max_q_len || P < 0 || P + T > a.max_blocks * 16) {
        if (lane == 0) flag_error(a.err, PA_DEVERR_BAD_LEN);
        return;
    }
    const uint64_t bits = a.mask[row];
    float q[E], acc[E], m = -INFINITY, l = 0.f;
    const float sl2 = a.scale * 1.4426950408889634f * (FP8 ? a.k_scale[kvh] : 1.f);
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[((size_t)row * a.Hq + h) * D + lane * E + e]);
        acc[e] = 0.f;
    }
    for (int t = 0; t < P + T; ++t) {
        if (t >= P && !((bits >> (t - P)) & 1)) continue;
        const int64_t blk = a.block_tables[(size_t)b * a.max_blocks + (t >> 4)];
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) flag_error(a.err, PA_DEVERR_BAD_BLOCK);
            continue;
        }
        const size_t at = ((blk * a.Hkv + kvh) * 16 + (t & 15)) * D + lane * E;
        float s = 0.f, v[E];
        for (int e = 0; e < E; ++e) {
            float k;
            if constexpr (FP8) {
                k = (float)static_cast<const __nv_fp8_e4m3 *>(a.k_cache)[at + e];
                v[e] = (float)static_cast<const __nv_fp8_e4m3 *>(a.v_cache)[at + e];
            } else {
                k = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.k_cache)[at + e]);
                v[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.v_cache)[at + e]);
            }
            s = fmaf(q[e], k, s);
        }
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= sl2;
        const float mn = fmaxf(m, s), al = mn == -INFINITY ? 1.f : ex2(m - mn), p = mn == -INFINITY ? 0.f : ex2(s - mn);
        m = mn;
        l = l * al + p;
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * al + p * v[e];
    }
    const float inv = (l > 0.f ? 1.f / l : 0.f) * (FP8 ? a.v_scale[kvh] : 1.f);
    for (int e = 0; e < E; ++e)
        static_cast<__nv_bfloat16 *>(a.out)[((size_t)row * a.Hq + h) * D + lane * E + e] = __float2bfloat16_rn(acc[e] * inv);
}

}  // namespace

size_t tree_ws_bytes(int) { return 0; }

cudaError_t launch_tree(const TreeArgs &a, void *, cudaStream_t st) {
    const dim3 grid((unsigned)(((long long)a.total_q * a.Hq + 3) / 4));
    if (a.D == 128) return launch_pdl(a.fp8 ? tree_kernel<128, true> : tree_kernel<128, false>, grid, dim3(128), 0, st, a);
    if (a.D == 64) return launch_pdl(a.fp8 ? tree_kernel<64, true> : tree_kernel<64, false>, grid, dim3(128), 0, st, a);
    return cudaErrorNotSupported;
}

}  // namespace pa
