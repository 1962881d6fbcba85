// sv_tree_mass.cu -- attention weight gathered by each slot of a paged cache:
// mass[p] += sum over the accepted nodes' rows r of exp(s_rp - lse_r).
//
// Simplest form: a warp for each (slot, key head), its key in registers, over
// the rows one after another.
#include <cuda_fp16.h>

#include "sv_common.cuh"
#include "sv_tree.h"

namespace sv {

namespace {

template <bool FP16>
__device__ __forceinline__ float2 pair_of(uint32_t w) {
    if (FP16) return __half22float2(*reinterpret_cast<__half2 *>(&w));
    return make_float2(bf16_lo(w), bf16_hi(w));
}

constexpr int kMassWarps = 8;

template <bool FP16, int D>
__global__ void __launch_bounds__(kMassWarps * 32) accumulate_kernel(const AccumParams P) {
    constexpr int W = D / 64;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.z, g = blockIdx.y;
    const int mn = P.t.max_nodes;
    const int n = P.n[b], nodes = P.t.nodes[b], L = P.lens[b];
    if (n < 0) return;
    int bad = 0;
    const int64_t row0 = P.t.row_off[b];
    if (nodes < 0 || nodes > mn || n >= nodes) bad |= SPECVERIFY_STATUS_BAD_TREE;
    else if (row0 < 0 || row0 > P.rows - nodes) bad |= SPECVERIFY_STATUS_BAD_ROW;
    if (L < 0 || !cache_holds(P.c, (int64_t)L + nodes)) bad |= SPECVERIFY_STATUS_BAD_CACHE;
    if (!bad) {
        int prev = -1;
        for (int i = 0; i <= n; ++i) {
            const int j = P.path[(int64_t)b * mn + i];
            if (j <= prev || j >= nodes) bad |= SPECVERIFY_STATUS_BAD_TREE;
            prev = j;
        }
        for (int i = threadIdx.x; i < (L + n) / P.c.page + 1; i += blockDim.x)
            if (page_at(P.c, b, i) < 0) bad |= SPECVERIFY_STATUS_BAD_CACHE;
    }
    if (bad) atomicOr(P.status, bad);
    if (__syncthreads_or(bad)) return;
    for (int s = blockIdx.x * kMassWarps + warp; s < L + n + 1; s += gridDim.x * kMassWarps) {
        const int64_t pg = page_of(P.c, b, s);
        const uint32_t *kr = reinterpret_cast<const uint32_t *>(
            P.c.k + pg * P.c.ps + (int64_t)g * P.c.hs + (int64_t)(s % P.c.page) * P.c.ts);
        float k[2 * W];
        for (int w = 0; w < W; ++w) {
            const float2 f = pair_of<FP16>(__ldg(kr + lane + 32 * w));
            k[2 * w] = f.x;
            k[2 * w + 1] = f.y;
        }
        float sum = 0.0f;
        for (int i = max(0, s - L); i <= n; ++i) {
            const int64_t row = row0 + P.path[(int64_t)b * mn + i];
            for (int hh = 0; hh < P.G; ++hh) {
                const int h = g * P.G + hh;
                const uint32_t *qr =
                    reinterpret_cast<const uint32_t *>(P.q + row * P.q_rs + h * P.q_hs);
                float x = 0.0f;
                for (int w = 0; w < W; ++w) {
                    const float2 f = pair_of<FP16>(__ldg(qr + lane + 32 * w));
                    x = fmaf(k[2 * w], f.x, fmaf(k[2 * w + 1], f.y, x));
                }
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                sum += exp2f(fmaf(x, P.scale_log2,
                                  -P.lse[row * P.heads + h] * 1.4426950408889634f));
            }
        }
        if (lane == 0)
            atomicAdd(&P.c.mass[pg * P.c.mps + g * P.c.mhs + (s % P.c.page) * P.c.mts], sum);
    }
}

}  // namespace

cudaError_t launch_accumulate(const AccumParams &p, int num_sms, cudaStream_t s) {
    (void)num_sms;
    const dim3 grid(64, p.c.kv_heads, p.t.B);
    if (p.c.fp16 && p.c.d == 128)
        accumulate_kernel<true, 128><<<grid, kMassWarps * 32, 0, s>>>(p);
    else if (p.c.fp16)
        accumulate_kernel<true, 64><<<grid, kMassWarps * 32, 0, s>>>(p);
    else if (p.c.d == 128)
        accumulate_kernel<false, 128><<<grid, kMassWarps * 32, 0, s>>>(p);
    else
        accumulate_kernel<false, 64><<<grid, kMassWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace sv
