// sv_tree_mass.cu -- attention weight gathered by each slot of a paged cache:
// mass[p] += sum over the accepted nodes' rows r of exp(s_rp - lse_r).
//
// The keys are read once, and with the few rows of an accepted path that read
// bounds the call. The product is turned over, S^T = K Q^T: a slot is a lane of
// tensor memory and a row a column, so the sum over the rows stays within a
// thread and needs no running maximum (the rows' logsumexps are known). A
// persistent CTA per SM:
//   warps 0-3, 4-7  two groups, every other tile of 128 slots each, a slot a
//                   thread: exponentials, their sum, one addition to mass;
//   warp 8          issues the products (one thread);
//   warp 9          copies K tiles into a ring of shared-memory slots;
//   warps 10, 11    gather the rows' queries and logsumexps a chunk ahead.
// (B = 24, 9 to 16 thousand tokens: 103 us, 6.1 TB/s, 90 % of the copy rate.)
// More than 128 rows are taken in chunks over the same tiles. A tile belongs to
// one group in every chunk, so a slot's chunks are added in order by one thread
// and the sum is the same every time.
#include <cuda_fp16.h>

#include "sv_tcgen05.cuh"
#include "sv_tree.h"

namespace sv {

namespace {

constexpr int kRows = 128;                 // of a chunk
constexpr int kMassThreads = 384;
constexpr int kGroupThreads = 128;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kScoutThreads = 64;
constexpr uint32_t kCols = 2 * kRows;      // tensor memory: S of both groups
constexpr int kHead = kMassHead;           // units of an item's start on the line (see below)

template <int D>
struct Shape {
    static constexpr int kPanel = kTile * 128;
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kSlots = D == 128 ? 5 : 10;
    static constexpr int kRing = 2 * kTileBytes;  // after the two Q tiles
    static constexpr int kMisc = kRing + kSlots * kTileBytes;
    static constexpr int kSmem = kMisc + 2048;
};

struct Misc {
    float lse[2][kRows];                   // of a chunk's rows, times log2(e)
    uint64_t full[10], empty[10], q_full[2], q_empty[2], s_full[2], s_empty[2], drain;
    int32_t b0, rest0;                     // the CTA's first sequence and unit in it
    uint32_t tmem;
    long long scan[kMassThreads / 32];
    int32_t abort;
    int32_t bad[2];                        // the chunk's sequence adds nothing
};
static_assert(sizeof(Misc) <= 2048, "Misc");

struct Seq {
    int L, n, tiles;                       // tiles 0: idle or bad
    int64_t row0;

    // (the host has checked that they fit 31 bits)
    __device__ int units(const AccumParams &P) const {
        return tiles ? (tiles + kHead) * P.c.kv_heads : 0;
    }
};

// The error of sequence b's sizes; its path and pages are the scouts' matter.
__device__ __forceinline__ int seq_error(const AccumParams &P, int b, const Seq &s) {
    if (s.n < 0) return 0;
    const int nodes = P.t.nodes[b];
    if (nodes < 0 || nodes > P.t.max_nodes || s.n >= nodes) return SPECVERIFY_STATUS_BAD_TREE;
    if (s.row0 < 0 || s.row0 > P.rows - nodes) return SPECVERIFY_STATUS_BAD_ROW;
    if (s.L < 0 || !cache_holds(P.c, (int64_t)s.L + s.n + 1)) return SPECVERIFY_STATUS_BAD_CACHE;
    return 0;
}

__device__ __forceinline__ Seq seq_of(const AccumParams &P, int b) {
    Seq s;
    s.n = P.n[b];
    s.L = P.lens[b];
    s.row0 = P.t.row_off[b];
    s.tiles = s.n >= 0 && seq_error(P, b, s) == 0 ? (s.L + s.n + kTile) / kTile : 0;
    return s;
}

// All (sequence, key head) items' tiles, kHead units for each item's start
// before them, form one line that is cut evenly over the CTAs.
struct Segment {
    Seq s;
    int b, head, tile0, n, rows, chunks;
};

struct Walk {
    int b;
    int rest;        // next unit within sequence b
    long long left;  // units of this CTA still to do

    __device__ bool next(const AccumParams &P, Segment &g) {
        while (left > 0) {
            g.s = seq_of(P, b);
            if (rest >= g.s.units(P)) {
                rest = 0;
                if (++b >= P.t.B) left = 0;  // (sizes that changed meanwhile)
                continue;
            }
            const int len = g.s.tiles + kHead;
            g.head = rest / len;
            const int u = rest - g.head * len;
            const int end = (int)min((long long)len, u + left);
            rest += end - u;
            left -= end - u;
            g.b = b;
            g.tile0 = max(u - kHead, 0);
            g.n = end - kHead - g.tile0;
            if (g.n <= 0) continue;
            g.rows = (g.s.n + 1) * P.G;
            g.chunks = (g.rows + kRows - 1) / kRows;
            return true;
        }
        return false;
    }
};

__device__ __forceinline__ bool wait_on(Misc &M, uint64_t &bar, uint32_t parity, const AccumParams &P) {
    return ::sv::wait_on(bar, parity, M.abort, P.status, P.wait_ns);
}

// ---------------------------------------------------------------------------

__device__ void sum_role(const AccumParams &P, Misc &M, Walk walk, uint32_t tmem) {
    const int tid = threadIdx.x, w = tid >> 7, lane_row = tid & 127;
    const uint32_t ts = tmem + ((uint32_t)(lane_row & ~31) << 16) + w * kRows;
    const float c2 = P.scale_log2;
    uint32_t chunk = 0, first = 0, phase = 0;  // first: tiles of the CTA's segments so far
    Segment g;
    while (walk.next(P, g)) {
        const int last = g.s.L + g.s.n;  // the last slot that gathers
        for (int q = 0; q < g.chunks; ++q, ++chunk) {
            const int rows = min(kRows, g.rows - q * kRows);
            const float *lse = M.lse[chunk & 1];
            bool ready = false;
            for (int j = (first ^ w) & 1; j < g.n; j += 2) {  // the same tiles in every chunk
                const int s = (g.tile0 + j) * kTile + lane_row;
                const int64_t page = s <= last ? page_of(P.c, g.b, s) : -1;
                if (!ready) {  // the scouts' lse and verdict
                    if (!wait_on(M, M.q_full[chunk & 1], chunk >> 1 & 1, P)) return;
                    ready = true;
                }
                if (!wait_on(M, M.s_full[w], phase, P)) return;
                phase ^= 1;
                tc_fence_after();
                // a slot that a node wrote is seen by the later ones only
                const int from = s > g.s.L ? (s - g.s.L) * P.G - q * kRows : 0;
                float sum[4] = {};
                for (int c0 = 0; c0 < rows; c0 += 32) {
                    uint32_t x[32];
                    tmem_ld32(ts + c0, x);
                    tmem_wait_ld();
                    if (c0 + 32 <= rows && (g.tile0 + j + 1) * kTile <= g.s.L) {
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 z = *reinterpret_cast<const float4 *>(lse + c0 + c);
                            sum[0] += ex2_approx(fmaf(__uint_as_float(x[c]), c2, -z.x));
                            sum[1] += ex2_approx(fmaf(__uint_as_float(x[c + 1]), c2, -z.y));
                            sum[2] += ex2_approx(fmaf(__uint_as_float(x[c + 2]), c2, -z.z));
                            sum[3] += ex2_approx(fmaf(__uint_as_float(x[c + 3]), c2, -z.w));
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (c0 + c < rows && c0 + c >= from)
                                sum[c & 3] += ex2_approx(fmaf(__uint_as_float(x[c]), c2, -lse[c0 + c]));
                    }
                }
                tc_fence_before();
                mbar_arrive(smem_u32(&M.s_empty[w]));
                if (page >= 0 && !M.bad[chunk & 1])
                    atomicAdd(&P.c.mass[page * P.c.mps + g.head * P.c.mhs +
                                        (int64_t)place_of(P.c, s).token * P.c.mts],
                              (sum[0] + sum[1]) + (sum[2] + sum[3]));
            }
            if (!ready && !wait_on(M, M.q_full[chunk & 1], chunk >> 1 & 1, P)) return;
            mbar_arrive(smem_u32(&M.q_empty[chunk & 1]));  // its lse is not read again
        }
        first += g.n;
    }
}

template <bool FP16, int D>
__device__ void mma_role(const AccumParams &P, Misc &M, char *smem, Walk walk, uint32_t tmem) {
    using Sh = Shape<D>;
    const uint32_t q0 = smem_u32(smem), ring = q0 + Sh::kRing;
    const bool on = elect_one();
    uint32_t chunk = 0, turn = 0, first = 0, uses[2] = {0, 0};
    Segment g;
    bool ok = true;
    while (ok && walk.next(P, g)) {
        for (int q = 0; ok && q < g.chunks; ++q, ++chunk) {
            const int rows = min(kRows, g.rows - q * kRows);
            const uint32_t desc = mma_desc(FP16, false, kTile, (rows + 15) / 16 * 16);
            ok = wait_on(M, M.q_full[chunk & 1], chunk >> 1 & 1, P);
            const uint32_t b = q0 + (chunk & 1) * Sh::kTileBytes;
            for (int j = 0; ok && j < g.n; ++j, ++turn) {
                const uint32_t slot = turn % Sh::kSlots, w = (first + j) & 1;
                ok = wait_on(M, M.full[slot], turn / Sh::kSlots & 1, P) &&
                     wait_on(M, M.s_empty[w], (uses[w]++ & 1) ^ 1, P);
                if (!ok) break;
                tc_fence_after();
                const uint32_t a = ring + slot * Sh::kTileBytes;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k >> 2) * Sh::kPanel + (k & 3) * 32;
                    mma_ss(tmem + w * kRows, smem_desc(a + off, 0), smem_desc(b + off, 0), desc, k > 0, on);
                }
                mma_commit(smem_u32(&M.s_full[w]), on);
                mma_commit(smem_u32(&M.empty[slot]), on);
            }
            if (ok) mma_commit(smem_u32(&M.q_empty[chunk & 1]), on);
        }
        first += g.n;
    }
    // No product, nor the arrival of one, outlives the CTA. Whoever reads the last ones
    // may have given up waiting for them, also where every wait of this warp was met.
    mma_commit(smem_u32(&M.drain), on);
    mbar_wait_bounded(smem_u32(&M.drain), 0);
}

template <int D>
__device__ void load_role(const AccumParams &P, const CUtensorMap *mk, Misc &M, char *smem,
                          Walk walk) {
    using Sh = Shape<D>;
    const int lane = threadIdx.x & 31, box = P.box;
    const uint32_t ring = smem_u32(smem) + Sh::kRing;
    uint32_t use = 0;
    Segment g;
    bool ok = true;
    while (ok && walk.next(P, g)) {
        const int len = g.s.L + g.s.n + 1;
        const auto page_id = [&](int j) -> int {  // of the lane's box in tile j, -1: none
            const int s = (g.tile0 + j) * kTile + lane * box;
            return j < g.n && lane * box < kTile && s < len ? (int)page_of(P.c, g.b, s) : -1;
        };
        for (int q = 0; ok && q < g.chunks; ++q) {
            int page = page_id(0);
            for (int j = 0; ok && j < g.n; ++j) {
                const int next = page_id(j + 1);
                const uint32_t slot = use % Sh::kSlots, bar = smem_u32(&M.full[slot]);
                ok = wait_on(M, M.empty[slot], (use / Sh::kSlots & 1) ^ 1, P);
                if (!ok) break;
                ++use;
                const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, page >= 0));
                if (lane == 0) mbar_arrive_expect_tx(bar, boxes * box * D * 2);
                __syncwarp();
                if (page >= 0) {
                    const int s = (g.tile0 + j) * kTile + lane * box;
                    const uint32_t dst = ring + slot * Sh::kTileBytes + lane * box * 128;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tile_load(dst + c * Sh::kPanel, mk, c * 64, place_of(P.c, s).token, g.head, page, bar);
                }
                __syncwarp();
                page = next;
            }
        }
    }
    // no copy outlives the CTA
    for (uint32_t u = use > Sh::kSlots ? use - Sh::kSlots : 0; u < use; ++u)
        mbar_wait_bounded(smem_u32(&M.full[u % Sh::kSlots]), u / Sh::kSlots & 1);
}

template <int D>
__device__ void scout_role(const AccumParams &P, Misc &M, char *smem, Walk walk) {
    using Sh = Shape<D>;
    constexpr int C = D / 8, R = kScoutThreads / C;  // 16-byte chunks of a row, rows at a time
    const int tid = threadIdx.x - (kMassThreads - kScoutThreads), c = tid % C;
    uint32_t chunk = 0;
    Segment g;
    bool ok = true;  // (the two warps meet at every segment, also one that gave up)
    while (walk.next(P, g)) {
        const int32_t *path = P.path + (int64_t)g.b * P.t.max_nodes;
        int bad = 0;
        {  // the path rises within the tree, the pages are the pool's
            const int nodes = P.t.nodes[g.b];
            for (int i = tid; i <= g.s.n; i += kScoutThreads) {
                const int j = path[i], prev = i > 0 ? path[i - 1] : -1;
                if (j <= prev || j >= nodes) bad |= SPECVERIFY_STATUS_BAD_TREE;
            }
            const int pages = place_of(P.c, g.s.L + g.s.n).index + 1;
#pragma unroll 8
            for (int i = tid; i < pages; i += kScoutThreads)
                if (page_at(P.c, g.b, i) < 0) bad |= SPECVERIFY_STATUS_BAD_CACHE;
        }
        if (bad) atomicOr(P.status, bad);
        uint32_t any;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
            "barrier.cta.red.or.pred q, 2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(any)
            : "r"((uint32_t)bad)
            : "memory");
        for (int q = 0; q < g.chunks; ++q, ++chunk) {
            const int x = chunk & 1, rows = min(kRows, g.rows - q * kRows);
            ok = ok && wait_on(M, M.q_empty[x], (chunk >> 1 & 1) ^ 1, P);
            if (!ok) break;
            const uint32_t tile = smem_u32(smem) + x * Sh::kTileBytes + (c >> 3) * Sh::kPanel;
            // a bad path names no rows: its chunk is left as it is and not added
            const int dn = R / P.G, dh = R - dn * P.G, r0 = q * kRows + tid / C;
            int node = r0 / P.G, hh = r0 - node * P.G;
            for (int r = tid / C; r < rows && !any; r += R) {
                const char *src = P.q + (g.s.row0 + path[node]) * P.q_rs +
                                  (int64_t)(g.head * P.G + hh) * P.q_hs + c * 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 tile + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                             "l"(src)
                             : "memory");
                node += dn;
                hh += dh;
                if (hh >= P.G) {
                    hh -= P.G;
                    ++node;
                }
            }
            for (int r = tid; r < rows && !any; r += kScoutThreads) {
                const int i = (q * kRows + r) / P.G, h = g.head * P.G + (q * kRows + r) - i * P.G;
                M.lse[x][r] = P.lse[(g.s.row0 + path[i]) * P.heads + h] * 1.4426950408889634f;
            }
            if (tid == 0) M.bad[x] = (int32_t)any;
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            mbar_arrive(smem_u32(&M.q_full[x]));
        }
    }
}

template <bool FP16, int D>
__global__ void __launch_bounds__(kMassThreads, 1)
    accumulate_kernel(const __grid_constant__ AccumParams P, const __grid_constant__ CUtensorMap mk) {
    using Sh = Shape<D>;
    extern __shared__ __align__(1024) char smem[];
    Misc &M = *reinterpret_cast<Misc *>(smem + Sh::kMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < Sh::kSlots; ++i) {
            mbar_init(smem_u32(&M.full[i]), 1);
            mbar_init(smem_u32(&M.empty[i]), 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_u32(&M.q_full[w]), kScoutThreads);
            mbar_init(smem_u32(&M.q_empty[w]), 1 + 2 * kGroupThreads);
            mbar_init(smem_u32(&M.s_full[w]), 1);
            mbar_init(smem_u32(&M.s_empty[w]), kGroupThreads);
        }
        mbar_init(smem_u32(&M.drain), 1);
        M.abort = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) tmem_alloc(smem_u32(&M.tmem), kCols);
    after_previous();

    // the line: each thread a run of sequences, a scan over the threads
    const int per = (P.t.B + kMassThreads - 1) / kMassThreads;
    const int b0 = min(P.t.B, tid * per), b1 = min(P.t.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        const Seq s = seq_of(P, b);
        mine += s.units(P);
        if (s.tiles == 0 && s.n >= 0 && blockIdx.x == 0) atomicOr(P.status, seq_error(P, b, s));
    }
    long long incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) M.scan[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long before = incl - mine, total = 0;
    for (int i = 0; i < kMassThreads / 32; ++i) {
        if (i < warp) before += M.scan[i];
        total += M.scan[i];
    }
    const Cut cut(total, gridDim.x);
    const int cta = min((int)blockIdx.x, cut.ctas);
    const long long lo = cut.at(cta), hi = cut.at(min(cta + 1, cut.ctas));
    if (lo < hi && before <= lo && lo < before + mine) {
        long long at = before;
        for (int b = b0; b < b1; ++b) {
            const long long n = seq_of(P, b).units(P);
            if (lo < at + n) {
                M.b0 = b;
                M.rest0 = (int)(lo - at);
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    const Walk walk{M.b0, M.rest0, hi - lo};
    const uint32_t tmem = M.tmem;
    if (warp < kMmaWarp) {
        sum_role(P, M, walk, tmem);
    } else if (warp == kMmaWarp) {
        mma_role<FP16, D>(P, M, smem, walk, tmem);
    } else if (warp == kLoadWarp) {
        load_role<D>(P, &mk, M, smem, walk);
    } else {
        scout_role<D>(P, M, smem, walk);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_free(tmem, kCols);
}

template <bool FP16, int D>
cudaError_t launch(const AccumParams &p, const CUtensorMap &mk, int ctas, cudaStream_t s) {
    return launch_after(accumulate_kernel<FP16, D>, dim3((unsigned)ctas), kMassThreads,
                        Shape<D>::kSmem, s, 1, p, mk);
}

template <bool FP16, int D>
cudaError_t prepare() {
    return cudaFuncSetAttribute(accumulate_kernel<FP16, D>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem);
}

}  // namespace

cudaError_t prepare_accumulate() {
    cudaError_t e = prepare<false, 64>();
    if (e == cudaSuccess) e = prepare<false, 128>();
    if (e == cudaSuccess) e = prepare<true, 64>();
    if (e == cudaSuccess) e = prepare<true, 128>();
    return e;
}

cudaError_t launch_accumulate(AccumParams p, int num_sms, cudaStream_t s) {
    CUtensorMap mk;
    p.box = cache_box(p.c.page);
    if (!cache_map(p.c, p.c.k, p.box, &mk)) return cudaErrorInvalidValue;
    if (p.c.fp16)
        return p.c.d == 128 ? launch<true, 128>(p, mk, num_sms, s) : launch<true, 64>(p, mk, num_sms, s);
    return p.c.d == 128 ? launch<false, 128>(p, mk, num_sms, s)
                        : launch<false, 64>(p, mk, num_sms, s);
}

}  // namespace sv
