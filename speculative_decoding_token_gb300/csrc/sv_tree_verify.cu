// sv_tree_verify.cu -- greedy verify of a token tree: the exact-match walk
// (the Kadimisetty notes, "Greedy vs sampling": a draft is kept while it is
// the target's argmax) along the branches of a tree.
//
// Only the rows on the accepted path decide, about two of a tree's dozens, so
// the walk reads those alone, one after another, and is bound by the latency
// of n + 1 dependent row reads: a cluster of kCtas CTAs per sequence reads
// each row, CTA c the columns [c per, (c + 1) per), tells the others its first
// maximum through distributed shared memory, and every CTA takes the same step.
#include "sv_rows.cuh"
#include "sv_tree.h"

namespace sv {

namespace {

constexpr int kVtCtas = 8;
constexpr int kVtThreads = 256;
constexpr int kVtWarps = kVtThreads / 32;
constexpr int kVtBatch = 5;  // 16-byte loads of a thread in flight

// a before b: the larger value, then the lower index; a NaN before all
__device__ __forceinline__ void take_first(float &best, int32_t &idx, float ob, int32_t oi) {
    const bool take = (ob != ob) ? true
                      : (best != best) ? false
                      : (oi >= 0 && (idx < 0 || ob > best || (ob == best && oi < idx)));
    if (take) {
        best = ob;
        idx = oi;
    }
}

template <int DT>
__global__ void __launch_bounds__(kVtThreads, 4) tree_verify_kernel(const TreeVerifyParams P) {
    __shared__ __align__(16) float4 s_slice[2][kVtCtas];
    __shared__ float2 s_warp[kVtWarps];
    __shared__ int32_t s_parent[kMaxNodes], s_token[kMaxNodes], s_path[kMaxNodes];
    constexpr int PV = DT == SV_DT_FP32 ? 4 : 8;  // logits in a 16-byte vector
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
    for (;;) {  // at most `nodes` steps: each goes to a later node
        const char *row = P.target + (row0 + node) * P.stride_bytes;
        // the first child's slice on its way to L2: where the walk goes on, it is
        // usually there
        if (warp == kVtWarps - 1) {
            int child = -1;
            for (int j0 = (node + 1) & ~31; j0 < nodes && child < 0; j0 += 32) {
                const int j = j0 + lane;
                const uint32_t hit =
                    __ballot_sync(0xffffffffu, j > node && j < nodes && s_parent[j] == node);
                if (hit) child = j0 + __ffs(hit) - 1;
            }
            if (child >= 0 && v1 > v0 && lane == 0)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                 P.target + (row0 + child) * P.stride_bytes + v0 * 16),
                             "r"((uint32_t)min((v1 - v0) * 16, (int64_t)1 << 18))
                             : "memory");
        }
        const uint4 *rv = reinterpret_cast<const uint4 *>(row);
        float best = -INFINITY;
        int32_t idx = -1;
        for (int64_t vi0 = v0 + threadIdx.x; vi0 < v1; vi0 += kVtBatch * kVtThreads) {
            uint4 v[kVtBatch];
#pragma unroll
            for (int i = 0; i < kVtBatch; ++i)
                if (vi0 + i * kVtThreads < v1) v[i] = __ldg(rv + vi0 + i * kVtThreads);
#pragma unroll
            for (int i = 0; i < kVtBatch; ++i) {
                const int64_t vi = vi0 + i * kVtThreads;
                if (vi >= v1) break;
                const float m = vec_max<DT>(v[i]);
                if (m != m || m > best || idx < 0) {  // later indexes: a tie keeps the first
                    if (best == best) {
                        float f[PV];
                        vec_floats<DT>(v[i], f);
                        int e = 0;
#pragma unroll
                        for (int j = PV - 1; j >= 0; --j)
                            if (f[j] == m) e = j;
                        best = m;
                        idx = (int32_t)(vi * PV + e);
                    }
                }
            }
        }
        for (int64_t e = v1 * PV + threadIdx.x; e < c1; e += kVtThreads)  // the ragged end at V
            take_first(best, idx, load_logit<DT>(row, e), (int32_t)e);
        const float2 r = warp_combine_greedy(best, idx);
        if (lane == 0) s_warp[warp] = r;
        if (n == 0) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        __syncthreads();
        if (warp == 0) {
            best = lane < kVtWarps ? s_warp[lane].x : -INFINITY;
            idx = lane < kVtWarps ? __float_as_int(s_warp[lane].y) : -1;
            const float2 c = warp_combine_greedy(best, idx);
            if (lane < kVtCtas)
                st_cluster_f4(cluster_addr(&s_slice[n & 1][rank], (uint32_t)lane),
                              make_float4(c.x, c.y, 0.0f, 0.0f));
        }
        // The barrier orders the slices, and step n + 2 reuses this step's only
        // after every CTA has passed the barrier of step n + 1.
        cluster_sync();
        best = -INFINITY;
        idx = -1;
#pragma unroll
        for (int c = 0; c < kVtCtas; ++c)
            take_first(best, idx, s_slice[n & 1][c].x, __float_as_int(s_slice[n & 1][c].y));
        pick = idx;
        nan = best != best;
        if (nan) break;
        if (threadIdx.x == 0) s_path[n] = node;
        // the lowest child with that token (every warp for itself)
        int next = -1;
        for (int j0 = (node + 1) & ~31; j0 < nodes && next < 0; j0 += 32) {
            const int j = j0 + lane;
            const uint32_t hit = __ballot_sync(
                0xffffffffu, j > node && j < nodes && s_parent[j] == node && s_token[j] == pick);
            if (hit) next = j0 + __ffs(hit) - 1;
        }
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.t.B * kVtCtas));
    cfg.blockDim = dim3(kVtThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kVtCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (dtype == SPECVERIFY_FP32)
        return cudaLaunchKernelEx(&cfg, tree_verify_kernel<SV_DT_FP32>, p);
    return cudaLaunchKernelEx(&cfg, tree_verify_kernel<SV_DT_BF16>, p);
}

}  // namespace sv
