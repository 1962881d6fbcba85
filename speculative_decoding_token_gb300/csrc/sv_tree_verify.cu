// sv_tree_verify.cu -- greedy verify of a token tree: the exact-match walk
// (the Kadimisetty notes, "Greedy vs sampling": a draft is kept while it is
// the target's argmax) along the branches of a tree.
//
// Only the rows on the accepted path decide, about two of a tree's dozens, so
// the walk reads those alone, one after another, and is bound by the latency
// of n + 1 dependent row reads: a cluster of kVtCtas CTAs per sequence reads
// each row, CTA c the columns [c per, (c + 1) per), every warp tells all of
// them its first maximum through distributed shared memory, and every CTA takes
// the same step: 1.8 us (V = 152064; B = 64, 4 to 48 nodes: 21 us a call).
#include "sv_rows.cuh"
#include "sv_tree.h"

namespace sv {

namespace {

constexpr int kVtCtas = 8;
constexpr int kVtThreads = 256;
constexpr int kVtWarps = kVtThreads / 32;
constexpr int kVtBatch = 10;  // 16-byte vectors that a thread holds

// A load that is issued where it stands, ahead of the barriers before its use.
__device__ __forceinline__ uint4 ld_early(const void *p) {
    uint4 x;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "l"(p));
    return x;
}

// A candidate of the argmax: order-preserving bits of its value (-0 as +0, a NaN
// above all), and its index. The larger value wins, then the lower index.
__device__ __forceinline__ uint32_t value_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void warp_best(uint32_t &key, uint32_t &idx) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, key);
    idx = __reduce_min_sync(0xffffffffu, key == top ? idx : 0xffffffffu);
    key = top;
}

__device__ __forceinline__ void st_cluster_u2(uint32_t addr, uint32_t x, uint32_t y) {
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}

template <int DT>
__device__ __forceinline__ float logit_at(const char *row, int64_t v) {
    if (DT == SV_DT_FP32) return reinterpret_cast<const float *>(row)[v];
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[v] << 16);
}

template <int DT>
__global__ void __launch_bounds__(kVtThreads, 3) tree_verify_kernel(const __grid_constant__ TreeVerifyParams P) {
    __shared__ __align__(16) uint2 s_slice[2][kVtCtas * kVtWarps];  // every warp's candidate
    __shared__ int32_t s_parent[kMaxNodes], s_token[kMaxNodes], s_path[kMaxNodes];
    constexpr int PV = DT == SV_DT_FP32 ? 4 : 8;  // logits in a 16-byte vector
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank();
    const int b = blockIdx.x / kVtCtas;
    const int mn = P.t.max_nodes;
    int32_t *tok = P.tok_out + (int64_t)b * mn, *path = P.path_out + (int64_t)b * mn;

    // validation (every CTA, the same answer)
    const int nodes = P.t.nodes[b];
    int bad = 0;
    int64_t row0 = 0;
    if (nodes < 0 || nodes > mn) {
        bad = SPECVERIFY_STATUS_BAD_TREE;
    } else if (nodes > 0) {
        row0 = P.t.row_off[b];
        if (row0 < 0 || row0 > P.rows - nodes) bad = SPECVERIFY_STATUS_BAD_ROW;
    }
    int bad_parent = 0, bad_token = 0;
    if (bad == 0 && (int)threadIdx.x < nodes) {
        const int j = threadIdx.x;
        const int32_t up = P.t.parent[(int64_t)b * mn + j], x = P.t.tokens[(int64_t)b * mn + j];
        s_parent[j] = up;
        s_token[j] = x;
        bad_parent = j == 0 ? up != -1 : (up < 0 || up >= j);
        bad_token = j > 0 && (x < 0 || (int64_t)x >= P.V);
    }
    if (__syncthreads_or(bad_parent)) bad |= SPECVERIFY_STATUS_BAD_TREE;
    if (__syncthreads_or(bad_token)) bad |= SPECVERIFY_STATUS_BAD_TOKEN;
    if (bad || nodes == 0) {
        if (rank == 0) {
            for (int i = threadIdx.x; i < mn; i += kVtThreads) tok[i] = path[i] = -1;
            if (threadIdx.x == 0) {
                P.n_out[b] = -1;
                if (bad) atomicOr(P.status, bad);
            }
        }
        return;  // every CTA of the cluster leaves here
    }

    // no CTA's shared memory is written before that CTA runs (waited for below)
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");

    // this CTA's columns: whole vectors, the last CTA's ending at V
    const int64_t per = ((P.V + kVtCtas - 1) / kVtCtas + PV - 1) / PV * PV;
    const int64_t c0 = min(P.V, (int64_t)rank * per), c1 = min(P.V, c0 + per);
    const int64_t v0 = c0 / PV, v1 = c1 / PV;
    int node = 0, n = 0;
    int32_t pick = -1;
    bool nan = false;
    // Where the target agrees with a draft it is mostly the first child's, so that
    // child's row is on its way (into registers as far as they reach, the rest
    // to L2) while the cluster decides the step.
    uint4 v[kVtBatch];
    const auto fetch = [&](int to) {
        const char *row = P.target + (row0 + to) * P.stride_bytes;
#pragma unroll
        for (int i = 0; i < kVtBatch; ++i) {
            const int64_t vi = v0 + threadIdx.x + i * kVtThreads;
            if (vi < v1) v[i] = ld_early(row + vi * 16);
        }
    };
    const int64_t beyond = v0 + kVtBatch * kVtThreads;  // vectors that registers do not hold
    fetch(0);
    for (;;) {  // at most `nodes` steps: each goes to a later node
        const char *row = P.target + (row0 + node) * P.stride_bytes;
        const uint4 *rv = reinterpret_cast<const uint4 *>(row);
        uint32_t key = 0, idx = 0xffffffffu;
        {
            // the maximum of the held vectors, then the first vector and element of it
            float m[kVtBatch], best = -INFINITY;
#pragma unroll
            for (int i = 0; i < kVtBatch; ++i) {
                const int64_t vi = v0 + threadIdx.x + i * kVtThreads;
                m[i] = vi < v1 ? vec_max<DT>(v[i]) : -INFINITY;
                best = max_nan(best, m[i]);
            }
            uint4 x = v[0];
            int at = 0;
#pragma unroll
            for (int i = kVtBatch - 1; i >= 0; --i)
                if (m[i] == best && v0 + threadIdx.x + i * kVtThreads < v1) {
                    at = i;
                    x = v[i];
                }
            if (v0 + threadIdx.x < v1) {
                float f[PV];
                vec_floats<DT>(x, f);
                int e = 0;
#pragma unroll
                for (int j = PV - 1; j >= 0; --j)
                    if (f[j] == best) e = j;
                key = value_key(best);
                idx = (uint32_t)((v0 + threadIdx.x + at * kVtThreads) * PV + e);
            }
        }
#pragma unroll 4
        for (int64_t vi = beyond + threadIdx.x; vi < v1; vi += kVtThreads) {
            const uint4 x = rv[vi];
            const float m = vec_max<DT>(x);
            if (value_key(m) > key) {  // later indexes: a tie keeps the first
                float f[PV];
                vec_floats<DT>(x, f);
                int e = 0;
#pragma unroll
                for (int j = PV - 1; j >= 0; --j)
                    if (f[j] == m) e = j;
                key = value_key(m);
                idx = (uint32_t)(vi * PV + e);
            }
        }
        for (int64_t e = v1 * PV + threadIdx.x; e < c1; e += kVtThreads) {  // the ragged end at V
            const uint32_t k = value_key(logit_at<DT>(row, e));
            if (k > key || idx == 0xffffffffu) {
                key = k;
                idx = (uint32_t)e;
            }
        }
        // the lowest child (of the token `want`, if that is not -1), every warp for itself
        const auto child_of = [&](int32_t want) {
            int found = -1;
            for (int j0 = (node + 1) & ~31; j0 < nodes && found < 0; j0 += 32) {
                const int j = j0 + lane;
                const uint32_t hit =
                    __ballot_sync(0xffffffffu, j > node && j < nodes && s_parent[j] == node &&
                                                   (want < 0 || s_token[j] == want));
                if (hit) found = j0 + __ffs(hit) - 1;
            }
            return found;
        };
        const int guess = child_of(-1);
        if (guess >= 0) {
            fetch(guess);
            if (beyond < v1 && threadIdx.x == 0)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                 P.target + (row0 + guess) * P.stride_bytes + beyond * 16),
                             "r"((uint32_t)min((v1 - beyond) * 16, (int64_t)1 << 18))
                             : "memory");
        }
        warp_best(key, idx);
        if (n == 0) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        if (lane < kVtCtas)
            st_cluster_u2(cluster_addr(&s_slice[n & 1][rank * kVtWarps + warp], (uint32_t)lane), key,
                          idx);
        // The barrier orders the candidates, and step n + 2 reuses this step's only
        // after every CTA has passed the barrier of step n + 1.
        cluster_sync();
        static_assert(kVtCtas * kVtWarps == 64, "two candidates a lane");
        const uint2 a = s_slice[n & 1][lane], z = s_slice[n & 1][lane + 32];
        const bool second = z.x > a.x || (z.x == a.x && z.y < a.y);
        key = second ? z.x : a.x;
        idx = second ? z.y : a.y;
        warp_best(key, idx);
        pick = (int32_t)idx;
        nan = key == 0xffffffffu;
        if (nan) break;
        if (threadIdx.x == 0) s_path[n] = node;
        const int next = child_of(pick);
        if (next >= 0 && next != guess) fetch(next);
        if (next < 0) break;
        node = next;
        ++n;
    }
    if (rank == 0) {
        __syncthreads();
        for (int i = threadIdx.x; i < mn; i += kVtThreads) {
            path[i] = !nan && i <= n ? s_path[i] : -1;
            tok[i] = nan || i > n ? -1 : (i == n ? pick : s_token[s_path[i + 1]]);
        }
        if (threadIdx.x == 0) {
            P.n_out[b] = nan ? -1 : n;
            if (nan) atomicOr(P.status, SPECVERIFY_STATUS_BAD_LOGIT);
        }
    }
}

}  // namespace

cudaError_t launch_tree_verify(const TreeVerifyParams &p, int dtype, cudaStream_t s) {
    const dim3 grid((unsigned)(p.t.B * kVtCtas));
    if (dtype == SPECVERIFY_FP32)
        return launch_after(tree_verify_kernel<SV_DT_FP32>, grid, kVtThreads, 0, s, kVtCtas, p);
    return launch_after(tree_verify_kernel<SV_DT_BF16>, grid, kVtThreads, 0, s, kVtCtas, p);
}

}  // namespace sv
