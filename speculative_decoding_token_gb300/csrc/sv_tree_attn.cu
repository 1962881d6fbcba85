// sv_tree_attn.cu -- attention of a tree of drafted tokens over a paged cache.
//
// Simplest form: a warp for each (node, query head), the head's elements over
// its lanes, one slot after another with the running maximum and sum of the
// softmax (Milakov and Gimelshein, "Online normalizer calculation for
// softmax"). Every row reads its keys for itself, so it is bound by
// instructions, far from the cache's bytes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_common.cuh"
#include "sv_tree.h"

namespace sv {

namespace {

template <bool FP16>
__device__ __forceinline__ float2 to_float2(uint32_t w) {
    if (FP16) return __half22float2(*reinterpret_cast<__half2 *>(&w));
    return make_float2(bf16_lo(w), bf16_hi(w));
}

template <bool FP16>
__device__ __forceinline__ uint32_t from_float2(float a, float b) {
    if (FP16) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}

constexpr int kRowWarps = 4;

template <bool FP16, int D>
__global__ void __launch_bounds__(kRowWarps * 32) tree_attn_kernel(const TreeAttnParams P) {
    constexpr int W = D / 64;  // 32-bit words of a row in a lane
    __shared__ uint32_t s_mask[kMaskWords];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.z, j = blockIdx.y, h = blockIdx.x * kRowWarps + warp;
    const int mn = P.t.max_nodes;
    const int nodes = P.t.nodes[b];
    int bad = 0;
    if (nodes < 0 || nodes > mn) bad = SPECVERIFY_STATUS_BAD_TREE;
    const int64_t row0 = bad ? 0 : P.t.row_off[b];
    if (!bad && nodes > 0 && (row0 < 0 || row0 > P.rows - nodes)) bad = SPECVERIFY_STATUS_BAD_ROW;
    if (bad || j >= nodes) {
        if (bad && threadIdx.x == 0) atomicOr(P.status, bad);
        return;
    }
    const int L = P.lens[b];
    if (L < 0 || !cache_holds(P.c, (int64_t)L + nodes)) bad = SPECVERIFY_STATUS_BAD_CACHE;
    for (int i = 0; i < nodes; ++i) {
        const int up = P.t.parent[(int64_t)b * mn + i];
        if (i == 0 ? up != -1 : (up < 0 || up >= i)) bad |= SPECVERIFY_STATUS_BAD_TREE;
    }
    for (int i = threadIdx.x; i < kMaskWords; i += blockDim.x) s_mask[i] = 0;
    __syncthreads();
    if (!bad && threadIdx.x == 0)
        for (int i = j; i >= 0; i = P.t.parent[(int64_t)b * mn + i])
            s_mask[i >> 5] |= 1u << (i & 31);
    __syncthreads();
    if (h >= P.heads) return;
    const int64_t row = row0 + j;
    const uint32_t *qr = reinterpret_cast<const uint32_t *>(P.q + row * P.q_rs + h * P.q_hs);
    float q[2 * W], o[2 * W];
    for (int w = 0; w < W; ++w) {
        const float2 f = to_float2<FP16>(qr[lane + 32 * w]);
        q[2 * w] = f.x;
        q[2 * w + 1] = f.y;
        o[2 * w] = o[2 * w + 1] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    const int64_t head = (int64_t)(h / P.G) * P.c.hs;
    for (int s = 0; s < L + nodes && !bad; ++s) {
        if (s >= L && !(s_mask[(s - L) >> 5] >> ((s - L) & 31) & 1)) continue;
        const int64_t pg = page_of(P.c, b, s);
        if (pg < 0) {
            bad = SPECVERIFY_STATUS_BAD_CACHE;
            break;
        }
        const int64_t off = pg * P.c.ps + head + (int64_t)(s % P.c.page) * P.c.ts;
        const uint32_t *kr = reinterpret_cast<const uint32_t *>(P.c.k + off);
        const uint32_t *vr = reinterpret_cast<const uint32_t *>(P.c.v + off);
        float x = 0.0f;
        for (int w = 0; w < W; ++w) {
            const float2 f = to_float2<FP16>(__ldg(kr + lane + 32 * w));
            x = fmaf(q[2 * w], f.x, fmaf(q[2 * w + 1], f.y, x));
        }
        for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
        x *= P.scale_log2;
        const float mn2 = fmaxf(m, x);
        const float keep = exp2f(m - mn2), p = exp2f(x - mn2);
        m = mn2;
        l = l * keep + p;
        for (int w = 0; w < W; ++w) {
            const float2 f = to_float2<FP16>(__ldg(vr + lane + 32 * w));
            o[2 * w] = fmaf(p, f.x, o[2 * w] * keep);
            o[2 * w + 1] = fmaf(p, f.y, o[2 * w + 1] * keep);
        }
    }
    if (bad && lane == 0) atomicOr(P.status, bad);
    const float inv = bad ? NAN : 1.0f / l;
    uint32_t *orow = reinterpret_cast<uint32_t *>(P.out + row * P.o_rs + h * P.o_hs);
    for (int w = 0; w < W; ++w)
        orow[lane + 32 * w] = from_float2<FP16>(o[2 * w] * inv, o[2 * w + 1] * inv);
    if (P.lse && lane == 0)
        P.lse[row * P.heads + h] = bad ? NAN : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t prepare_tree() { return cudaSuccess; }

cudaError_t launch_tree_attention(const TreeAttnParams &p, int num_sms, cudaStream_t s) {
    (void)num_sms;
    const dim3 grid((p.heads + kRowWarps - 1) / kRowWarps, p.t.max_nodes, p.t.B);
    if (p.c.fp16 && p.c.d == 128)
        tree_attn_kernel<true, 128><<<grid, kRowWarps * 32, 0, s>>>(p);
    else if (p.c.fp16)
        tree_attn_kernel<true, 64><<<grid, kRowWarps * 32, 0, s>>>(p);
    else if (p.c.d == 128)
        tree_attn_kernel<false, 128><<<grid, kRowWarps * 32, 0, s>>>(p);
    else
        tree_attn_kernel<false, 64><<<grid, kRowWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace sv
