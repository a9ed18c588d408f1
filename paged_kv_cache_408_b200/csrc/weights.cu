// weights.cu -- a decode step that also adds every cached token's attention
// weight to a running sum kept beside the cache.
//
// out as in pa_decode; for token t of sequence b, kv head k:
//     w[slot(b, t)][k] = (t < seen[b] ? w : 0) + sum_{h in group k} p_h(t),
//     p_h(t) = 2^(s_h(t) - L_h),  s = scale log2(e) q_h . k_t,
//     L_h the log2-sum-exp of s_h over the sequence.
//
// Two kernels: one warp per (sequence, query head) attends and leaves L_h;
// then one warp per (sequence, kv head, block) computes the scores again.
#include "common.cuh"
#include "kernels.h"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <int E, bool FP8>
PA_DEVICE void load_dims(const void *cache, size_t at, float (&x)[E]) {
    for (int e = 0; e < E; ++e) {
        if constexpr (FP8) x[e] = (float)static_cast<const __nv_fp8_e4m3 *>(cache)[at + e];
        else x[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(cache)[at + e]);
    }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(128) attend_kernel(const DecodeArgs a, float *lse) {
    constexpr int E = D / 32;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (long long)a.B * a.Hq) return;
    const int b = (int)(row / a.Hq), h = (int)(row % a.Hq), kvh = h / (a.Hq / a.Hkv);
    int len = a.seq_lens[b];
    if (len < 0 || len > a.max_blocks * 16) {
        if (lane == 0) flag_error(a.err, PA_DEVERR_BAD_LEN);
        len = 0;
    }
    float q[E], acc[E], m = -INFINITY, l = 0.f;
    const float sl2 = a.scale * kLog2e * (FP8 ? a.k_scale[kvh] : 1.f);
    load_dims<E, false>(a.q, row * D + lane * E, q);
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int t = 0; t < len; ++t) {
        const int64_t blk = a.block_tables[(size_t)b * a.max_blocks + (t >> 4)];
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) flag_error(a.err, PA_DEVERR_BAD_BLOCK);
            continue;
        }
        const size_t at = ((blk * a.Hkv + kvh) * 16 + (t & 15)) * D + lane * E;
        float k[E], v[E], s = 0.f;
        load_dims<E, FP8>(a.k_cache, at, k);
        load_dims<E, FP8>(a.v_cache, at, v);
        for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= sl2;
        const float mn = fmaxf(m, s), al = mn == -INFINITY ? 1.f : ex2(m - mn), p = mn == -INFINITY ? 0.f : ex2(s - mn);
        m = mn;
        l = l * al + p;
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * al + p * v[e];
    }
    const float inv = (l > 0.f ? 1.f / l : 0.f) * (FP8 ? a.v_scale[kvh] : 1.f);
    for (int e = 0; e < E; ++e)
        static_cast<__nv_bfloat16 *>(a.out)[row * D + lane * E + e] = __float2bfloat16_rn(acc[e] * inv);
    if (lane == 0) lse[row] = l > 0.f ? m + log2f(l) : INFINITY;  // no token: every weight 2^-inf = 0
}

template <int D, bool FP8>
__global__ void __launch_bounds__(128) add_kernel(const DecodeArgs a, const float *lse, float *w, const int32_t *seen) {
    constexpr int E = D / 32;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, G = a.Hq / a.Hkv;
    const long long u = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int j = (int)(u % a.max_blocks), kvh = (int)(u / a.max_blocks % a.Hkv), b = (int)(u / a.max_blocks / a.Hkv);
    if (b >= a.B) return;
    const int len = a.seq_lens[b];
    if (len > a.max_blocks * 16 || j * 16 >= len) return;
    const int64_t blk = a.block_tables[(size_t)b * a.max_blocks + j];
    if (blk < 0 || blk >= a.num_blocks) return;
    const float sl2 = a.scale * kLog2e * (FP8 ? a.k_scale[kvh] : 1.f);
    const int old = seen ? seen[b] : len;
    for (int i = 0; i < 16 && j * 16 + i < len; ++i) {
        const size_t slot = (blk * a.Hkv + kvh) * 16 + i;
        float k[E], sum = 0.f;
        load_dims<E, FP8>(a.k_cache, slot * D + lane * E, k);
        for (int g = 0; g < G; ++g) {
            const size_t row = (size_t)b * a.Hq + kvh * G + g;
            float q[E], s = 0.f;
            load_dims<E, false>(a.q, row * D + lane * E, q);
            for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            sum += exp2f(s * sl2 - lse[row]);
        }
        if (lane == 0) w[slot] = (j * 16 + i < old ? w[slot] : 0.f) + sum;
    }
}

template <int D, bool FP8>
cudaError_t run(const DecodeArgs &a, float *weights, const int32_t *seen, float *lse, cudaStream_t st) {
    const long long rows = (long long)a.B * a.Hq, blocks = (long long)a.B * a.Hkv * a.max_blocks;
    cudaError_t e = launch_pdl(attend_kernel<D, FP8>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, a, lse);
    if (e != cudaSuccess) return e;
    return launch_pdl(add_kernel<D, FP8>, dim3((unsigned)((blocks + 3) / 4)), dim3(128), 0, st, a, (const float *)lse,
                      weights, seen);
}

}  // namespace

size_t weights_ws_bytes(int B, int Hq, int, int, int) { return (size_t)B * Hq * sizeof(float); }

cudaError_t launch_decode_weights(const DecodeArgs &a, float *weights, const int32_t *seen, void *workspace,
                                  cudaStream_t st) {
    float *lse = static_cast<float *>(workspace);
    if (a.D == 128) return a.fp8 ? run<128, true>(a, weights, seen, lse, st) : run<128, false>(a, weights, seen, lse, st);
    if (a.D == 64) return a.fp8 ? run<64, true>(a, weights, seen, lse, st) : run<64, false>(a, weights, seen, lse, st);
    return cudaErrorNotSupported;
}

}  // namespace pa
