// sv_tree_cache.cu -- what a paged cache keeps: the commit of an accepted path
// and the eviction of the tokens that gathered the least attention weight.
#include "sv_tree.h"

namespace sv {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// ---------------------------------------------------------------------------
// Commit. Slot L + i takes slot L + path[i]: path rises, so path[i] >= i, and
// what entry i overwrites no later entry reads. A thread owns 16 bytes of one
// (layer, head) of k or of v for the whole path and reads a group of entries
// before it writes them. Bound by the latency of those dependent loads.
constexpr int kCommitThreads = 256;
constexpr int kCommitGroup = 4;

__global__ void __launch_bounds__(kCommitThreads) commit_kernel(const CommitParams P) {
    __shared__ int64_t s_src[kMaxNodes], s_dst[kMaxNodes];   // byte offset of the slot, head 0
    __shared__ int64_t s_mass[kMaxNodes];                    // element offset of L + i
    const int b = blockIdx.x, layer = blockIdx.y;
    const int L = P.lens[b], n = P.n[b];
    const CacheParams &c = P.c;
    int bad = 0;
    if (n >= P.max_nodes) bad = SPECVERIFY_STATUS_BAD_TREE;
    int64_t src = 0, dst = 0, mass = 0;
    if (n >= 0 && !bad) {
        if (L < 0) bad = SPECVERIFY_STATUS_BAD_CACHE;
        const int i = threadIdx.x;
        if (!bad && i <= n) {
            const int32_t *path = P.path + (int64_t)b * P.max_nodes;
            const int j = path[i], prev = i > 0 ? path[i - 1] : -1;
            if (j <= prev || j >= P.max_nodes || (i == 0 && j != 0)) {
                bad = SPECVERIFY_STATUS_BAD_TREE;
            } else if (!cache_holds(c, (int64_t)L + j + 1)) {
                bad = SPECVERIFY_STATUS_BAD_CACHE;
            } else {
                const int64_t ps = page_of(c, b, L + j), pd = page_of(c, b, L + i);
                if (ps < 0 || pd < 0) bad = SPECVERIFY_STATUS_BAD_CACHE;
                src = ps * c.ps + (L + j) % c.page * c.ts;
                dst = pd * c.ps + (L + i) % c.page * c.ts;
                mass = pd * c.mps + (L + i) % c.page * c.mts;
                s_src[i] = src;
                s_dst[i] = dst;
                s_mass[i] = mass;
            }
        }
    }
    // bits of every thread: a bad path outranks a bad cache in the report
    const int bad_tree = __syncthreads_or(bad & SPECVERIFY_STATUS_BAD_TREE);
    bad = __syncthreads_or(bad) ? (bad_tree ? SPECVERIFY_STATUS_BAD_TREE
                                            : SPECVERIFY_STATUS_BAD_CACHE)
                                : 0;
    const bool move = n >= 0 && !bad;
    if (layer == 0 && threadIdx.x == 0) {
        P.new_lens[b] = L + (move ? n + 1 : 0);
        if (P.new_seen) P.new_seen[b] = P.seen[b] + (move ? n + 1 : 0);
        if (bad) atomicOr(P.status, bad);
    }
    if (!move) return;
    int first = 1;  // entries before it are in place
    while (first <= n && s_src[first] == s_dst[first]) ++first;
    const int chunks = c.d / 8;  // 16 bytes each
    for (int t = threadIdx.x; t < c.kv_heads * chunks * 2 && first <= n; t += kCommitThreads) {
        const int kv = t / (c.kv_heads * chunks), r = t % (c.kv_heads * chunks);
        char *base = (kv ? c.v : c.k) + layer * c.ls + r / chunks * c.hs + r % chunks * 16;
        for (int i = first; i <= n; i += kCommitGroup) {
            uint4 x[kCommitGroup];
#pragma unroll
            for (int e = 0; e < kCommitGroup; ++e)
                if (i + e <= n) x[e] = *reinterpret_cast<const uint4 *>(base + s_src[i + e]);
#pragma unroll
            for (int e = 0; e < kCommitGroup; ++e)
                if (i + e <= n) *reinterpret_cast<uint4 *>(base + s_dst[i + e]) = x[e];
        }
    }
    if (c.mass || c.pos) {
        for (int t = threadIdx.x; t < c.kv_heads * (n + 1); t += kCommitThreads) {
            const int i = t / c.kv_heads;
            const int64_t at = layer * c.mls + t % c.kv_heads * c.mhs + s_mass[i];
            if (c.mass) c.mass[at] = 0.0f;
            if (c.pos) c.pos[at] = P.seen[b] + i;
        }
    }
}

// ---------------------------------------------------------------------------
// Eviction, selection: one CTA for each (layer, sequence, key head). The
// budget-th largest key by a radix select over the keys' bits, most
// significant first, then the kept slots by counting in slot order.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBits = 8;
constexpr int kSelBins = 1 << kSelBits;

// Order-preserving bits of a mass: -0 as +0, a NaN as the least. A protected
// token's key is above every one of them.
__device__ __forceinline__ uint32_t mass_key(float m) {
    if (m != m) return 0u;
    const uint32_t u = __float_as_uint(m + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Item {
    int b, head, layer;
    int len, seen;
    int64_t base;  // of mass and pos, elements
};

__device__ __forceinline__ int64_t slot_at(const CacheParams &c, const Item &it, int s) {
    const int64_t pg = __ldg(&c.table[(int64_t)it.b * c.table_stride + s / c.page]);
    return it.base + pg * c.mps + (int64_t)(s % c.page) * c.mts;
}

__device__ __forceinline__ uint32_t key_of(const EvictParams &P, const Item &it, int s) {
    const int64_t at = slot_at(P.c, it, s);
    const int pos = P.c.pos[at];
    if (pos < P.sink || pos >= it.seen - P.recent) return 0xffffffffu;
    return mass_key(P.c.mass[at]);
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictParams P) {
    __shared__ uint32_t s_hist[kSelBins];
    __shared__ uint32_t s_pick[2];
    __shared__ int s_cnt[3][kSelWarps];
    const CacheParams &c = P.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = blockIdx.x;
    Item it;
    it.head = item % c.kv_heads;
    it.b = item / c.kv_heads % P.B;
    it.layer = item / c.kv_heads / P.B;
    it.len = P.lens[it.b];
    it.seen = P.seen[it.b];
    it.base = it.layer * c.mls + it.head * c.mhs;
    int bad = it.len < 0 || !cache_holds(c, it.len);
    if (!bad)
        for (int i = threadIdx.x; i < (it.len + c.page - 1) / c.page; i += kSelThreads)
            bad |= page_at(c, it.b, i) < 0;
    bad = __syncthreads_or(bad);
    const int N = it.len, keep = min(N, P.budget);
    if (threadIdx.x == 0) {
        if (P.moves > 0 && (N <= P.budget || bad)) P.move_cnt[item] = 0;
        if (it.layer == 0 && it.head == 0) P.new_lens[it.b] = bad ? N : keep;
        if (bad) atomicOr(P.status, SPECVERIFY_STATUS_BAD_CACHE);
    }
    if (bad) return;
    const bool copy = P.mass_out != c.mass, copy_pos = P.pos_out != c.pos;
    if (N <= P.budget) {
        if (copy || copy_pos)
            for (int s = threadIdx.x; s < N; s += kSelThreads) {
                const int64_t at = slot_at(c, it, s);
                if (copy) P.mass_out[at] = c.mass[at];
                if (copy_pos) P.pos_out[at] = c.pos[at];
            }
        return;
    }
    // the keep-th largest key: `prefix` its leading bits, `need` its rank among those that share them
    uint32_t prefix = 0, mask = 0;
    int need = keep;
    for (int shift = 32 - kSelBits; shift >= 0; shift -= kSelBits) {
        for (int i = threadIdx.x; i < kSelBins; i += kSelThreads) s_hist[i] = 0;
        __syncthreads();
        for (int s = threadIdx.x; s < N; s += kSelThreads) {
            const uint32_t k = key_of(P, it, s);
            if ((k & mask) == prefix) atomicAdd(&s_hist[k >> shift & (kSelBins - 1)], 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int left = need, bin = kSelBins - 1;
            for (; bin > 0 && (int)s_hist[bin] < left; --bin) left -= (int)s_hist[bin];
            s_pick[0] = (uint32_t)bin;
            s_pick[1] = (uint32_t)left;
        }
        __syncthreads();
        prefix |= s_pick[0] << shift;
        mask |= (uint32_t)(kSelBins - 1) << shift;
        need = (int)s_pick[1];
        __syncthreads();
    }
    // kept: keys above it, and the first `need` slots that equal it. Warp w owns
    // a run of slots; counts before it come from the other warps' totals.
    const int run = ((N + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int r0 = min(N, warp * run), r1 = min(N, r0 + run);
    int eq = 0;
    for (int s0 = r0; s0 < r1; s0 += 32) {
        const int s = s0 + lane;
        eq += __popc(__ballot_sync(kAll, s < r1 && key_of(P, it, s) == prefix));
    }
    if (lane == 0) s_cnt[0][warp] = eq;
    __syncthreads();
    int eq0 = 0;
    for (int w = 0; w < warp; ++w) eq0 += s_cnt[0][w];
    int holes = 0, movers = 0;
    const uint32_t below = (1u << lane) - 1u;
    for (int pass = 0; pass < 2; ++pass) {
        int e = eq0, hole = 0, mover = 0;
        if (pass == 1)
            for (int w = 0; w < warp; ++w) {
                hole += s_cnt[1][w];
                mover += s_cnt[2][w];
            }
        for (int s0 = r0; s0 < r1; s0 += 32) {
            const int s = s0 + lane;
            const uint32_t k = s < r1 ? key_of(P, it, s) : 0u;
            const uint32_t same = __ballot_sync(kAll, s < r1 && k == prefix);
            const bool kept =
                s < r1 && (k > prefix || (k == prefix && e + __popc(same & below) < need));
            e += __popc(same);
            const uint32_t hm = __ballot_sync(kAll, s < keep && s < r1 && !kept);
            const uint32_t mm = __ballot_sync(kAll, s >= keep && kept);
            if (pass == 1) {
                const int64_t list = (int64_t)item * P.moves;
                if (hm >> lane & 1) P.move_dst[list + hole + __popc(hm & below)] = s;
                if (mm >> lane & 1) P.move_src[list + mover + __popc(mm & below)] = s;
                if (kept && s < keep && (copy || copy_pos)) {
                    const int64_t at = slot_at(c, it, s);
                    if (copy) P.mass_out[at] = c.mass[at];
                    if (copy_pos) P.pos_out[at] = c.pos[at];
                }
            }
            hole += __popc(hm);
            mover += __popc(mm);
        }
        if (pass == 0) {
            if (lane == 0) {
                s_cnt[1][warp] = hole;
                s_cnt[2][warp] = mover;
            }
            __syncthreads();
        } else {
            holes = hole;
            movers = mover;
        }
    }
    (void)holes;
    if (warp == kSelWarps - 1 && lane == 0) P.move_cnt[item] = movers;
}

// Eviction, moves: a source lies at or past the budget and a destination
// below it, so moves never meet. A group of d / 8 threads takes one move.
constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams P) {
    const CacheParams &c = P.c;
    const int chunks = c.d / 8, item = blockIdx.x;
    const int head = item % c.kv_heads, b = item / c.kv_heads % P.B,
              layer = item / c.kv_heads / P.B;
    const int cnt = P.move_cnt[item];
    const int part = threadIdx.x % chunks;
    const int per = kMoveThreads / chunks;
    const int64_t base = layer * c.ls + head * c.hs + part * 16;
    for (int r = blockIdx.y * per + threadIdx.x / chunks; r < cnt; r += gridDim.y * per) {
        const int64_t list = (int64_t)item * P.moves + r;
        const int s = P.move_src[list], d = P.move_dst[list];
        const int64_t ps = __ldg(&c.table[(int64_t)b * c.table_stride + s / c.page]);
        const int64_t pd = __ldg(&c.table[(int64_t)b * c.table_stride + d / c.page]);
        const int64_t so = base + ps * c.ps + (int64_t)(s % c.page) * c.ts;
        const int64_t dof = base + pd * c.ps + (int64_t)(d % c.page) * c.ts;
        const uint4 k = *reinterpret_cast<const uint4 *>(c.k + so);
        const uint4 v = *reinterpret_cast<const uint4 *>(c.v + so);
        *reinterpret_cast<uint4 *>(c.k + dof) = k;
        *reinterpret_cast<uint4 *>(c.v + dof) = v;
        if (part < 2) {
            const int64_t mb = layer * c.mls + head * c.mhs;
            const int64_t ms = mb + ps * c.mps + (int64_t)(s % c.page) * c.mts;
            const int64_t md = mb + pd * c.mps + (int64_t)(d % c.page) * c.mts;
            if (part == 0)
                P.mass_out[md] = c.mass[ms];
            else
                P.pos_out[md] = c.pos[ms];
        }
    }
}

}  // namespace

cudaError_t launch_tree_commit(const CommitParams &p, cudaStream_t s) {
    commit_kernel<<<dim3(p.B, p.c.layers), kCommitThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_evict(const EvictParams &p, cudaStream_t s) {
    const int items = p.c.layers * p.B * p.c.kv_heads;
    evict_select_kernel<<<items, kSelThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.moves == 0) return e;
    evict_move_kernel<<<dim3(items, 32), kMoveThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace sv
