// sv_tree_cache.cu -- what a paged cache keeps: the commit of an accepted path
// and the eviction of the tokens that gathered the least attention weight.
#include <algorithm>

#include "sv_tree.h"

namespace sv {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// ---------------------------------------------------------------------------
// Commit. Slot L + i takes slot L + path[i]: path rises, so path[i] >= i, and
// what entry i overwrites no later entry reads. A thread owns 16 bytes of one
// (layer, head) of k or of v for the whole path and reads a group of entries
// before it writes them. A small call is bound by its three dependent loads (2.4 us;
// B = 64, one layer: 3.3). A batch of all layers is between them and its bytes: B =
// 64, 24 layers, of about 350 entries 250 that move, 50 MB read and written, 12.9 us,
// 3.8 TB/s (of 1536 CTAs 1216 fit at once, and each plans its sequence anew); 24
// layers more add 10.3 us, 5.4 TB/s, which is what rows of 256 bytes move at.
constexpr int kCommitThreads = 256;
constexpr int kCommitGroup = 4;

__global__ void __launch_bounds__(kCommitThreads) commit_kernel(const __grid_constant__ CommitParams P) {
    __shared__ int64_t s_src[kMaxNodes], s_dst[kMaxNodes];   // byte offset of the slot, head 0
    __shared__ int64_t s_mass[kMaxNodes];                    // element offset of L + i
    after_previous();
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
                src = ps * c.ps + place_of(c, L + j).token * c.ts;
                dst = pd * c.ps + place_of(c, L + i).token * c.ts;
                mass = pd * c.mps + place_of(c, L + i).token * c.mts;
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
// Eviction, selection: one CTA for each (layer, sequence, key head). Every slot
// becomes a 32-bit key, read once into shared memory while they fit (kKeyCap of
// them; beyond that the passes read mass and pos again, from L2). The budget-th
// largest key by a radix select, 11, 11 and 10 bits, most significant first;
// then the kept slots by counting in slot order. Bound by the instructions of the
// passes over the keys (20 to 33 thousand slots: 30 us) and, for a few thousand
// slots, by the latency of its dozen barriers (8 us).
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;             // two a thread
constexpr int kKeyCap = 48 * 1024;         // 192 KiB
constexpr int kSelBatch = 8;               // slots of a thread read at a time

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
    const Place p = place_of(c, s);
    const int64_t pg = c.table[(int64_t)it.b * c.table_stride + p.index];
    return it.base + pg * c.mps + (int64_t)p.token * c.mts;
}

__device__ __forceinline__ uint32_t key_of_token(const EvictParams &P, const Item &it, float mass,
                                                 int pos) {
    return pos < P.sink || pos >= it.seen - P.recent ? 0xffffffffu : mass_key(mass);
}

// Eviction, moves: a source lies at or past the budget and a destination below
// it, so moves never meet. d / 8 threads take a group of moves, all of its rows
// in flight at once; bound by the bytes of the moved rows. Four moves a group
// in the moving kernel (B = 16, 32k to 4k: 119 us a call; two 122, eight 151),
// two where the selecting CTA moves (its threads have 64 registers).
constexpr int kMoveThreads = 256;
constexpr int kMoveGroup = 4, kOwnGroup = 2;

// Moves of an item, groups `first`, `first` + `step`, ... by d / 8 threads, of
// which this is number `part`.
template <int M>
__device__ __forceinline__ void move_tokens(const EvictParams &P, int item, int cnt, int first,
                                            int step, int part) {
    const CacheParams &c = P.c;
    const int head = item % c.kv_heads, b = item / c.kv_heads % P.B,
              layer = item / c.kv_heads / P.B;
    const int64_t base = layer * c.ls + head * c.hs + part * 16;
    const int64_t mbase = layer * c.mls + head * c.mhs, list = (int64_t)item * P.moves;
    const int32_t *table = c.table + (int64_t)b * c.table_stride;
    for (int r0 = first * M; r0 < cnt; r0 += step * M) {
        int s[M], d[M];
        int64_t ps[M], pd[M];
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int64_t at = list + min(r0 + i, cnt - 1);
            s[i] = P.move_src[at];
            d[i] = P.move_dst[at];
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const Place a = place_of(c, s[i]), z = place_of(c, d[i]);
            ps[i] = table[a.index];
            pd[i] = table[z.index];
            s[i] = a.token;
            d[i] = z.token;
        }
        uint4 k[M], v[M];
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int64_t so = base + ps[i] * c.ps + s[i] * c.ts;
            k[i] = *reinterpret_cast<const uint4 *>(c.k + so);
            v[i] = *reinterpret_cast<const uint4 *>(c.v + so);
        }
        // thread `part` also takes mass or pos of one of the moves
        const int mi = part >> 1;
        if (mi < M && r0 + mi < cnt) {
            int64_t ms = 0, md = 0;
#pragma unroll
            for (int i = 0; i < M; ++i)
                if (i == mi) {
                    ms = mbase + ps[i] * c.mps + s[i] * c.mts;
                    md = mbase + pd[i] * c.mps + d[i] * c.mts;
                }
            if (part & 1)
                P.pos_out[md] = c.pos[ms];
            else
                P.mass_out[md] = c.mass[ms];
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            if (r0 + i >= cnt) break;
            const int64_t to = base + pd[i] * c.ps + d[i] * c.ts;
            *reinterpret_cast<uint4 *>(c.k + to) = k[i];
            *reinterpret_cast<uint4 *>(c.v + to) = v[i];
        }
    }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams P) {
    after_previous();
    const int chunks = P.c.d / 8, groups = kMoveThreads / chunks, item = blockIdx.x;
    move_tokens<kMoveGroup>(P, item, P.move_cnt[item], blockIdx.y * groups + threadIdx.x / chunks,
                gridDim.y * groups, threadIdx.x % chunks);
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const __grid_constant__ EvictParams P) {
    extern __shared__ uint32_t s_key[];
    __shared__ uint32_t s_hist[kSelBins];
    __shared__ int s_pick[2];
    __shared__ int s_cnt[3][kSelWarps];
    after_previous();
    const CacheParams &c = P.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
        for (int i = tid; i < (it.len + c.page - 1) / c.page; i += kSelThreads)
            bad |= page_at(c, it.b, i) < 0;
    for (int i = tid; i < kSelBins; i += kSelThreads) s_hist[i] = 0;
    bad = __syncthreads_or(bad);
    const int N = it.len, keep = min(N, P.budget);
    if (tid == 0) {
        if (!P.inline_moves && (N <= P.budget || bad)) P.move_cnt[item] = 0;
        if (it.layer == 0 && it.head == 0) P.new_lens[it.b] = bad ? N : keep;
        if (bad) atomicOr(P.status, SPECVERIFY_STATUS_BAD_CACHE);
    }
    if (bad) return;
    const bool copy = P.mass_out != c.mass, copy_pos = P.pos_out != c.pos;
    if (N <= P.budget) {
        if (copy || copy_pos)
            for (int s = tid; s < N; s += kSelThreads) {
                const int64_t at = slot_at(c, it, s);
                if (copy) P.mass_out[at] = c.mass[at];
                if (copy_pos) P.pos_out[at] = c.pos[at];
            }
        return;
    }
    const bool held = N <= kKeyCap;
    const auto key_of = [&](int s) {
        if (held) return s_key[s];
        const int64_t at = slot_at(c, it, s);
        return key_of_token(P, it, c.mass[at], c.pos[at]);
    };
    // the keep-th largest key: `prefix` its leading bits, `need` its rank among
    // those that share them
    uint32_t prefix = 0;
    int need = keep;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        const uint32_t bins = pass == 2 ? 1024u : 2048u;
        if (pass == 0) {
            for (int s0 = tid; s0 < N; s0 += kSelThreads * kSelBatch) {
                float m[kSelBatch];
                int pos[kSelBatch];
                int64_t at[kSelBatch];
#pragma unroll
                for (int i = 0; i < kSelBatch; ++i) {
                    at[i] = slot_at(c, it, min(s0 + i * kSelThreads, N - 1));
                    m[i] = c.mass[at[i]];
                    pos[i] = c.pos[at[i]];
                }
#pragma unroll
                for (int i = 0; i < kSelBatch; ++i) {
                    const int s = s0 + i * kSelThreads;
                    if (s >= N) break;
                    const uint32_t k = key_of_token(P, it, m[i], pos[i]);
                    if (held) s_key[s] = k;
                    atomicAdd(&s_hist[k >> shift], 1u);
                    if (s < keep) {  // what moves into a freed slot comes after, in the other kernel
                        if (copy) P.mass_out[at[i]] = m[i];
                        if (copy_pos) P.pos_out[at[i]] = pos[i];
                    }
                }
            }
        } else {
            const int above = pass == 1 ? 21 : 10;
            for (int s = tid; s < N; s += kSelThreads) {
                const uint32_t k = key_of(s);
                if (k >> above == prefix >> above) atomicAdd(&s_hist[k >> shift & (bins - 1)], 1u);
            }
        }
        __syncthreads();
        // keys in the bins above this thread's two (thread 0 has the highest)
        const int hi = (int)bins - 1 - 2 * tid;
        const int n1 = hi >= 0 ? (int)s_hist[hi] : 0, n0 = hi >= 1 ? (int)s_hist[hi - 1] : 0;
        int incl = n0 + n1;
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) s_cnt[0][warp] = incl;
        __syncthreads();
        int before = incl - n0 - n1;
        {
            const int t = s_cnt[0][lane];
            before += __reduce_add_sync(kAll, lane < warp ? t : 0);
        }
        if (before < need && need <= before + n1) {
            s_pick[0] = hi;
            s_pick[1] = need - before;
        } else if (before + n1 < need && need <= before + n1 + n0) {
            s_pick[0] = hi - 1;
            s_pick[1] = need - before - n1;
        }
        if (hi >= 0) s_hist[hi] = 0;
        if (hi >= 1) s_hist[hi - 1] = 0;
        __syncthreads();
        prefix |= (uint32_t)s_pick[0] << shift;
        need = s_pick[1];
    }
    // kept: keys above it, and the first `need` slots that equal it. Warp w owns
    // a run of slots; counts before it come from the other warps' totals.
    const int run = ((N + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int r0 = min(N, warp * run), r1 = min(N, r0 + run);
    int eq = 0, low_above = 0, high_above = 0, low_eq = 0;
    for (int s0 = r0; s0 < r1; s0 += 32) {
        const int s = s0 + lane;
        const uint32_t k = s < r1 ? key_of(s) : 0u;
        eq += s < r1 && k == prefix;
        low_eq += s < keep && s < r1 && k == prefix;
        low_above += s < keep && s < r1 && k > prefix;
        high_above += s >= keep && s < r1 && k > prefix;
    }
    eq = __reduce_add_sync(kAll, eq);
    low_eq = __reduce_add_sync(kAll, low_eq);
    low_above = __reduce_add_sync(kAll, low_above);
    high_above = __reduce_add_sync(kAll, high_above);
    if (lane == 0) s_cnt[0][warp] = eq;
    __syncthreads();
    const int eq0 = __reduce_add_sync(kAll, lane < warp ? s_cnt[0][lane] : 0);
    // of this warp's equal slots the first `take` are kept, those below the budget first
    const int take = max(0, min(eq, need - eq0)), low_take = min(take, low_eq);
    if (lane == 0) {
        s_cnt[1][warp] = max(0, min(r1, keep) - r0) - low_above - low_take;  // free slots
        s_cnt[2][warp] = high_above + take - low_take;                      // movers
    }
    __syncthreads();
    int hole = __reduce_add_sync(kAll, lane < warp ? s_cnt[1][lane] : 0);
    int mover = __reduce_add_sync(kAll, lane < warp ? s_cnt[2][lane] : 0);
    const uint32_t below = (1u << lane) - 1u;
    const int64_t list = (int64_t)item * P.moves;
    int e = eq0;
    for (int s0 = r0; s0 < r1; s0 += 32) {
        const int s = s0 + lane;
        const uint32_t k = s < r1 ? key_of(s) : 0u;
        const uint32_t same = __ballot_sync(kAll, s < r1 && k == prefix);
        const bool kept = s < r1 && (k > prefix || (k == prefix && e + __popc(same & below) < need));
        e += __popc(same);
        const uint32_t hm = __ballot_sync(kAll, s < keep && s < r1 && !kept);
        const uint32_t mm = __ballot_sync(kAll, s >= keep && kept);
        if (hm >> lane & 1) P.move_dst[list + hole + __popc(hm & below)] = s;
        if (mm >> lane & 1) P.move_src[list + mover + __popc(mm & below)] = s;
        hole += __popc(hm);
        mover += __popc(mm);
    }
    if (!P.inline_moves) {
        if (warp == kSelWarps - 1 && lane == 0) P.move_cnt[item] = mover;
        return;
    }
    if (warp == kSelWarps - 1 && lane == 0) s_pick[0] = mover;
    __syncthreads();
    const int chunks = c.d / 8;
    move_tokens<kOwnGroup>(P, item, s_pick[0], tid / chunks, kSelThreads / chunks, tid % chunks);
}

}  // namespace

cudaError_t launch_tree_commit(const CommitParams &p, cudaStream_t s) {
    return launch_after(commit_kernel, dim3(p.B, p.c.layers), kCommitThreads, 0, s, 1, p);
}

cudaError_t prepare_evict() {
    return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kKeyCap * (int)sizeof(uint32_t));
}

cudaError_t launch_evict(EvictParams p, cudaStream_t s) {
    const int items = p.c.layers * p.B * p.c.kv_heads;
    const int64_t capacity = (int64_t)p.c.max_pages * p.c.page;
    const int keys = (int)std::min<int64_t>(capacity, kKeyCap);
    // Up to a group of moves for each team of the selecting CTA are its own (B = 4,
    // 40 over 2048: 9.7 us against 10.8); a second kernel spreads more of them
    // over the SMs.
    p.inline_moves = p.moves <= kSelThreads / (p.c.d / 8) * kOwnGroup;
    const cudaError_t e = launch_after(evict_select_kernel, dim3((unsigned)items), kSelThreads,
                                       keys * sizeof(uint32_t), s, 1, p);
    if (e != cudaSuccess || p.inline_moves) return e;
    // blocks of an item: enough for its longest list, up to about four waves in all
    const int per = kMoveThreads / (p.c.d / 8) * kMoveGroup;
    const int most = (p.moves + per - 1) / per;
    return launch_after(evict_move_kernel,
                        dim3((unsigned)items, (unsigned)std::min(most, std::max(1, 8192 / items))),
                        kMoveThreads, 0, s, 1, p);
}

}  // namespace sv
