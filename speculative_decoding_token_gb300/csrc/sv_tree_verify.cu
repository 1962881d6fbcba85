// sv_tree_verify.cu -- greedy verify of a token tree: the exact-match walk
// (the Kadimisetty notes, "Greedy vs sampling": a draft is kept while it is
// the target's argmax) along the branches of a tree.
//
// Only the rows on the accepted path decide, about two of a tree's dozens, so
// the walk reads those alone, one after another, and is bound by the latency
// of n + 1 dependent row reads: a cluster of kVtCtas CTAs per sequence reads
// each row, CTA c the columns [c per, (c + 1) per), every warp sends all of them
// its first maximum (stores to distributed shared memory that count themselves
// on a barrier there: B = 16, V = 152064: 11.4 us a call; with a barrier of the
// cluster 12.7), and every CTA takes the same step, in about 1.8 us. B = 64, 4 to
// 48 nodes: 19.4 us; 57 sequences fit the GPU at a time. (Plain stores with a
// releasing arrival, which need no care where a wait runs out: 22.3 us.) Loading the first
// child's row ahead did not pay: where every cluster is at work it is traffic
// that many steps do not need.
#include "sv_rows.cuh"
#include "sv_tree.h"

namespace sv {

namespace {

constexpr int kVtCtas = 8;
constexpr int kVtThreads = 256;
constexpr int kVtWarps = kVtThreads / 32;
constexpr int kVtBatch = 10;  // 16-byte vectors that a thread loads at a time

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

// A store to another CTA's shared memory that counts its bytes on a barrier there.
__device__ __forceinline__ void send_u2(uint32_t addr, uint32_t bar, uint32_t x, uint32_t y) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(addr),
        "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// A wait for what other CTAs of the cluster send; gives up after `limit` nanoseconds.
__device__ __forceinline__ bool wait_sent(uint32_t bar, uint32_t parity, uint64_t limit) {
    const uint64_t t0 = global_ns();
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (global_ns() - t0 > limit) return false;
    }
}

// A plain store to another CTA's shared memory, there once both have passed a
// barrier of the cluster.
__device__ __forceinline__ void put_u1(uint32_t addr, int32_t x) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Waits for every candidate that was sent to this CTA, where warps of the cluster
// gave up: a store that counts itself must not meet a CTA that has left. A warp goes
// past a step only with all of its candidates, so every warp has sent those of the
// first `all` steps and some those of one step more; sent[w] is warp w's number, of
// this CTA's warp 0 `mine`. One thread.
__device__ __noinline__ void drain_sent(const int32_t *sent, int mine, const uint64_t *bars) {
    int all = sent[0], more = 0;
    for (int w = 1; w < kVtCtas * kVtWarps; ++w) all = min(all, sent[w]);
    for (int w = 0; w < kVtCtas * kVtWarps; ++w) more += sent[w] > all;
    mbar_wait_bounded(smem_u32(&bars[(all - 1) & 1]), (all - 1) >> 1 & 1);
    if (more == 0) return;
    const uint32_t bar = smem_u32(&bars[all & 1]), each = sizeof(uint2);
    if (mine > all)  // the barrier expects every warp's: count those that do not come
        asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar),
                     "r"((kVtCtas * kVtWarps - more) * each)
                     : "memory");
    else
        mbar_arrive_expect_tx(bar, more * each);
    mbar_wait_bounded(bar, all >> 1 & 1);
}

template <int DT>
__device__ __forceinline__ float logit_at(const char *row, int64_t v) {
    if (DT == SV_DT_FP32) return reinterpret_cast<const float *>(row)[v];
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[v] << 16);
}

template <int DT>
__global__ void __launch_bounds__(kVtThreads, 3) tree_verify_kernel(const __grid_constant__ TreeVerifyParams P) {
    // every warp's candidate, and its arrival, of the even and the odd steps
    __shared__ __align__(16) uint2 s_slice[2][kVtCtas * kVtWarps];
    __shared__ uint64_t s_bar[2];
    __shared__ int32_t s_late, s_sent[kVtCtas * kVtWarps];  // a warp of the cluster gave up; steps that it sent
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

    // no CTA's shared memory is written before that CTA has set it up (waited for below)
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&s_bar[0]), 1);
        mbar_init(smem_u32(&s_bar[1]), 1);
        s_late = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    cluster_arrive();

    // this CTA's columns: whole vectors, the last CTA's ending at V
    const int64_t per = ((P.V + kVtCtas - 1) / kVtCtas + PV - 1) / PV * PV;
    const int64_t c0 = min(P.V, (int64_t)rank * per), c1 = min(P.V, c0 + per);
    const int v0 = (int)(c0 / PV), v1 = (int)(c1 / PV);
    int node = 0, n = 0;
    int32_t pick = -1;
    bool nan = false, late = false;
    for (;;) {  // at most `nodes` steps: each goes to a later node
        const char *row = P.target + (row0 + node) * P.stride_bytes;
        // the thread's first vector of the largest element, then that element
        uint32_t key = 0, idx = 0xffffffffu;
        if (v0 + (int)threadIdx.x < v1) {
            float best = -INFINITY;
            int at = v0 + (int)threadIdx.x;
            bool odd = false;
            for (int from = at; from < v1; from += kVtBatch * kVtThreads) {
                uint4 v[kVtBatch];
#pragma unroll
                for (int i = 0; i < kVtBatch; ++i)
                    if (from + i * kVtThreads < v1)
                        v[i] = *reinterpret_cast<const uint4 *>(row + (int64_t)(from + i * kVtThreads) * 16);
#pragma unroll
                for (int i = 0; i < kVtBatch; ++i) {
                    if (from + i * kVtThreads >= v1) break;
                    const float m = vec_max<DT>(v[i]);
                    odd |= m != m;
                    if (m > best) {
                        best = m;
                        at = from + i * kVtThreads;
                    }
                }
            }
            float f[PV];
            vec_floats<DT>(*reinterpret_cast<const uint4 *>(row + (int64_t)at * 16), f);
            int e = 0;
#pragma unroll
            for (int j = PV - 1; j >= 0; --j)
                if (f[j] == best) e = j;
            key = odd ? 0xffffffffu : value_key(best);
            idx = (uint32_t)(at * PV + e);
        }
        for (int64_t e = (int64_t)v1 * PV + threadIdx.x; e < c1; e += kVtThreads) {  // the ragged end at V
            const uint32_t k = value_key(logit_at<DT>(row, e));
            if (k > key || idx == 0xffffffffu) {
                key = k;
                idx = (uint32_t)e;
            }
        }
        warp_best(key, idx);
        if (n == 0) cluster_wait();
        // Every CTA sends its candidates to all of them and waits for theirs on its
        // own barrier. Step n + 2 reuses step n's places: who is there has had this
        // CTA's candidates of step n + 1, sent after it had read step n's.
        const uint32_t bar = smem_u32(&s_bar[n & 1]);
        if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, sizeof(s_slice[0]));
        if (lane < kVtCtas)
            send_u2(cluster_addr(&s_slice[n & 1][rank * kVtWarps + warp], (uint32_t)lane),
                    cluster_addr(&s_bar[n & 1], (uint32_t)lane), key, idx);
        // (a warp leaves as a whole: its reductions are of all lanes)
        late = __any_sync(0xffffffffu, !wait_sent(bar, n >> 1 & 1, P.wait_ns));
        if (late) break;
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
    // nobody leaves while another may still send to it
    const int sent = n + 1;
    if (late && lane < kVtCtas) put_u1(cluster_addr(&s_late, (uint32_t)lane), 1);
    cluster_arrive();
    late = __syncthreads_or(late);
    if (rank == 0) {
        const bool none = nan || late;
        for (int i = threadIdx.x; i < mn; i += kVtThreads) {
            path[i] = !none && i <= n ? s_path[i] : -1;
            tok[i] = none || i > n ? -1 : (i == n ? pick : s_token[s_path[i + 1]]);
        }
        if (threadIdx.x == 0) {
            P.n_out[b] = none ? -1 : n;
            if (late) atomicOr(P.status, SPECVERIFY_STATUS_TIMEOUT);
            else if (nan) atomicOr(P.status, SPECVERIFY_STATUS_BAD_LOGIT);
        }
    }
    cluster_wait();
    if (*(volatile int32_t *)&s_late) {  // the same in every CTA
        if (lane < kVtCtas) put_u1(cluster_addr(&s_sent[rank * kVtWarps + warp], (uint32_t)lane), sent);
        cluster_arrive();
        cluster_wait();
        if (threadIdx.x == 0) drain_sent(s_sent, sent, s_bar);
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
