// sv_tree_attn.cu -- attention of a tree of drafted tokens over a paged cache,
// one pass over the keys and values with the running maximum and sum of the
// softmax (Milakov and Gimelshein, "Online normalizer calculation for
// softmax").
//
// The queries of a tree's nodes that share a key head are the rows of one
// matrix, row r = node r / G, head r % G, so each key is read once for all of
// them: S = Q K^T and O += P V run on the tensor core in tiles of 128 rows by
// 128 slots. A persistent CTA per SM:
//   warps 0-7, 8-15 two softmax groups, half a row a thread: S from tensor
//                   memory, P back to it, in two parts;
//   warp 16         issues the products;
//   warp 17         copies K and V tiles into a ring of shared-memory slots;
//   warps 18, 19    go ahead of them: the next segment's Q tiles, and the check
//                   of its pages and parents.
// The two groups take turns on the tensor core, one's softmax under the
// other's products. Up to 128 rows share one Q tile and the groups alternate
// over the slots' tiles (each with its own maximum, sum and O, joined at the
// end); more rows make two Q tiles, a group each, over the same slots.
//
// All (sequence, key head, block of rows) items' tiles of 128 slots, with a
// constant for each item's start, form one line that is cut evenly over the CTAs,
// first every sequence's first block of rows, then the second ones: where trees
// have two blocks, CTAs half the grid apart read the same keys at about the same
// time, and L2 serves one of them. An item cut in pieces leaves each piece's O
// (not yet divided), maximum and sum in the workspace, and a second kernel joins
// the pieces (3 us; the last of an item's CTAs joining them took longer, for its
// fence and counter); whole items are written directly.
//
// Up to 128 rows a key head the keys' bytes bound it: 1.39 us a tile of 64 KiB
// and CTA, 7.2 TB/s over 152 of them (B = 38, 65 thousand tokens each). With 256
// rows the products do: 88 cycles for each of nominally 64 in a trace (S = Q K^T
// reads 8 KiB of shared memory a product, all of the SM's bandwidth). B = 32, 64
// nodes, 64 heads over 8, 14 thousand tokens: 648 us in short bursts, 1.46 PFLOP/s;
// 726 us, 1.30 PFLOP/s, where calls follow one another for long and the 1400 W cap
// holds the clock at 1.70 GHz. Waits whose outcome is the whole warp's, and the
// uniform branches after them, are worth 5 % of that (683 us with a branch a lane).
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "sv_tcgen05.cuh"
#include "sv_tree.h"

namespace sv {

namespace {

constexpr int kSoftThreads = 512;
constexpr int kAttnThreads = kSoftThreads + 128;
constexpr int kMmaWarp = 16, kLoadWarp = 17, kScoutThreads = 64;
// A softmax thread holds half a row of S. A launch of 640 threads gives each 96
// registers; the groups draw 104 and the last warpgroup keeps 64 (104 * 512 +
// 64 * 128 registers, the launch's 96 * 640).
constexpr int kSoftRegs = 104, kOtherRegs = 64;
constexpr int kTmemCols = 512;
// The least weight of a piece, fp32's least number: keeps inf * weight infinite, and
// adds under 2^-21 where a finite piece (under 2^128) should count for nothing.
constexpr float kTiny = 0x1p-149f;

template <int D>
struct Shape {
    static constexpr int kPanel = kTile * 128;           // 64 elements of 128 rows
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kSlots = D == 128 ? 5 : 10;     // ring slots of a K or V tile
    static constexpr int kRing = 2 * kTileBytes;         // after the two Q tiles
    static constexpr int kMisc = kRing + kSlots * kTileBytes;
    static constexpr int kSmem = kMisc + 3 * 1024;
    // columns of tensor memory: S of both groups, then O of both; P lies over S
    static constexpr uint32_t kS = 0, kO = 2 * kTile;
};
static_assert(Shape<128>::kSmem <= 232448 && Shape<64>::kSmem <= 232448, "shared memory of a CTA");

// An item's place on the line starts with kHead units that are no tiles: what
// its start and end cost beside its tiles (queries, sums, the output).
// Six measured best over ragged batches (B = 16, 300 to 8000 tokens: 57.8 us;
// four 58.3, two 59.8, one 63.0).
constexpr int kHead = kAttnHead;

// What sequence b contributes to the line; 0 tiles: idle or bad.
struct Seq {
    int L, T, tiles, blocks;
    int64_t row0;

    // Units of the items of one block of rows (the host has checked that they fit 31 bits).
    __device__ int units(const TreeAttnParams &P, int block) const {
        return block < blocks ? (tiles + kHead) * P.c.kv_heads : 0;
    }
};

__device__ __forceinline__ int seq_error(const TreeAttnParams &P, int nodes, int64_t row0, int L) {
    if (nodes < 0 || nodes > P.t.max_nodes) return SPECVERIFY_STATUS_BAD_TREE;
    if (nodes == 0) return 0;
    if (row0 < 0 || row0 > P.rows - nodes) return SPECVERIFY_STATUS_BAD_ROW;
    if (L < 0 || !cache_holds(P.c, (int64_t)L + nodes)) return SPECVERIFY_STATUS_BAD_CACHE;
    return 0;
}

__device__ __forceinline__ Seq seq_of(const TreeAttnParams &P, int b) {
    Seq s;
    s.T = P.t.nodes[b];
    s.L = P.lens[b];
    s.row0 = P.t.row_off[b];
    s.tiles = s.blocks = 0;
    if (s.T != 0 && seq_error(P, s.T, s.row0, s.L) == 0) {
        s.tiles = (s.L + s.T + kTile - 1) / kTile;
        s.blocks = (s.T * P.G + 2 * kTile - 1) / (2 * kTile);
    }
    return s;
}

// A run of tiles of one item, all of a CTA's work in line order. Every role
// walks the same segments by itself.
struct Segment {
    Seq s;
    int b, head, block, tile0, n;
    int rows;      // of this item: up to 2 * kTile
    bool pair;     // two Q tiles
    bool first, last;  // holds the item's first, last tile
};

struct Walk {
    int b, block;
    int rest;         // next unit within sequence b's of that block
    long long left;   // units of this CTA still to do

    __device__ bool next(const TreeAttnParams &P, Segment &g) {
        while (left > 0) {
            g.s = seq_of(P, b);
            if (rest >= g.s.units(P, block)) {
                rest = 0;
                if (++b == P.t.B) {
                    b = 0;
                    if (++block >= P.blocks) left = 0;  // (sizes that changed meanwhile)
                }
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
            g.block = block;
            g.rows = min(g.s.T * P.G - g.block * 2 * kTile, 2 * kTile);
            g.pair = g.rows > kTile;
            g.first = g.tile0 == 0;
            g.last = g.tile0 + g.n == g.s.tiles;
            return true;
        }
        return false;
    }
};

// What the scouts say of a segment, and whoever clears its last values.
struct Scouted {
    Segment g;                             // n = 0: the CTA's work is done
    int8_t parent[kMaxNodes];
    uint32_t nonfinite[kMaskWords];        // nodes of it whose value has an inf or NaN
    uint32_t bad;                          // a page or a parent
};

struct Misc {
    float x[4][kTile];                     // what the halves and the groups tell each other of a row
    Scouted seg[2];                        // of the even and the odd segments
    uint64_t full[10], empty[10], q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2];
    uint64_t seg_full[2], seg_empty[2], begun, drain;  // begun: the first queries are there
    int32_t rest0;                         // the CTA's first unit in its first sequence,
    int32_t b0, block0;                    // that sequence, and the block of rows
    uint32_t tmem;
    long long scan[kAttnThreads / 32];
    int32_t abort;                         // a wait gave up
};
static_assert(sizeof(Misc) <= 3 * 1024, "Misc");

// Place of a segment's K and V tile j in the order of the ring's uses. Group w
// needs K of its next tile before V of its current one.
__device__ __forceinline__ uint32_t k_at(const Segment &g, int j) {
    return g.pair ? 2 * j : (j == 0 ? 0 : 2 * j - 1);
}
__device__ __forceinline__ uint32_t v_at(const Segment &g, int j) {
    return g.pair ? 2 * j + 1 : min(2 * j + 2, 2 * g.n - 1);
}

__device__ __forceinline__ bool wait_on(Misc &M, uint64_t &bar, uint32_t parity, const TreeAttnParams &P) {
    return ::sv::wait_on(bar, parity, M.abort, P.status, P.wait_ns);
}

// Barrier of the two softmax groups.
__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, 512;" ::: "memory"); }

// The same; whether every thread's v was true.
__device__ __forceinline__ bool soft_all(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 512, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

// Barrier of the scouts; whether every thread's v was true.
__device__ __forceinline__ bool scouts_all(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 10, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

// Barrier of the two warps that share 32 rows; whether any thread's v was true.
__device__ __forceinline__ bool pair_any(int bar, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(bar), "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    if (FP16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <bool FP16>
__device__ __forceinline__ float half_at(uint32_t w, int i) {
    const uint32_t x = (w >> (16 * i)) & 0xffffu;
    return FP16 ? __half2float(__ushort_as_half((unsigned short)x)) : __uint_as_float(x << 16);
}

// The halves of w that are inf or NaN, as a mask of their bits.
template <bool FP16>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) {
    constexpr uint32_t e = FP16 ? 0x7C00u : 0x7F80u;
    return ((w & e) == e ? 0xffffu : 0u) | (((w >> 16) & e) == e ? 0xffff0000u : 0u);
}

// 32 bytes, a whole sector of L2.
__device__ __forceinline__ void st_global_8(float *dst, const float *f) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(f[0]),
                 "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
}

// A weight is rounded to the cache's type (the product takes P in the type of V; as
// two terms, the rounding and the rest, P would double the products), off by at most
// half a step, 2^-8 or 2^-11 of itself. So an output is within that of the mean of
// |v| from the one of exact weights, before its own rounding of the same size: the
// error against 64 bits is 2.2e-3 of the outputs' size with bfloat16 (1.7e-3 for
// exact weights) and 2.2e-4 with binary16 (2.1e-4). The weight counts in the sum as
// it was before the rounding. It is relative to a reference maximum that
// is raised only when the running one passes it by kSlack binades (until then
// O and the sum need no rescaling). bfloat16 keeps fp32's range; binary16 has
// weights from 2^-24 to 2^16, so the reference's weight is 2^kShift there.
template <bool FP16>
struct Range {
    static constexpr float kSlack = FP16 ? 5.0f : 8.0f;
    static constexpr float kShift = FP16 ? 10.0f : 0.0f;
};

// ---------------------------------------------------------------------------
// softmax groups

template <bool FP16, int D>
__device__ void softmax_role(const TreeAttnParams &P, Misc &M, char *smem, uint32_t tmem) {
    using Sh = Shape<D>;
    constexpr int H = kTile / 2;               // columns of S that a thread holds
    constexpr int CW = D / 4;                  // columns of O at a time
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int w = warp >> 3, h = warp >> 2 & 1;  // group, half of its columns
    const int row = (warp & 3) * 32 + lane;    // of the group's Q tile
    const int pair_bar = 2 + w * 4 + (warp & 3);  // barrier of the two warps that share 32 rows
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + Sh::kS + w * kTile;
    const float c2 = P.scale_log2;
    const float ninf = -INFINITY;
    uint32_t s_phase = 0, o_phase = 0, seg = 0;  // o_phase: a bit for each group
    uint32_t base = 0;  // ring uses before this segment
    for (;; ++seg) {
        Scouted &sc = M.seg[seg & 1];
        // (the barrier: all have read the last segment's O and x)
        if (!soft_all(wait_on(M, M.seg_full[seg & 1], seg >> 1 & 1, P))) break;
        const Segment &g = sc.g;
        const int n = g.n;
        if (n == 0) break;
        const bool pair = g.pair;
        const int ahead = g.tile0 * kTile - g.s.L;
        // this thread's row
        const int r_item = (pair ? w * kTile : 0) + row;
        const int gr = g.block * 2 * kTile + min(r_item, g.rows - 1);
        const int node = gr / P.G, qh = g.head * P.G + gr - node * P.G;
        const bool warp_on = (pair ? w * kTile : 0) + (row & ~31) < g.rows;
        const bool mine = r_item < g.rows;  // (rows past the item's hold what the tile held before)
        float m_ref = ninf, l = 0.0f;
        bool fresh = true;
        int j = pair ? 0 : w;
        // A warp that gave up only keeps to the barriers of the others, to the next segment's start.
        const auto leave = [&] {
            for (; warp_on && j < n; j += pair ? 1 : 2)
                if (pair_any(pair_bar, false)) pair_any(pair_bar, false);
            for (int i = pair ? 1 : 3; i > 0; --i) soft_sync();
            soft_all(false);
        };
        for (; j < n; j += pair ? 1 : 2) {
            if (!wait_on(M, M.s_full[w], s_phase, P)) return leave();
            s_phase ^= 1;
            tc_fence_after();
            const int shift = ahead + j * kTile;  // column c is node c + shift, a token before 0
            const bool tail_tile = shift + kTile > 0;
            if (tail_tile && (!pair || w == 0)) {
                // a slot past the tree, or a node's inf or NaN: 0 in the products
                // (the latter are added where they are seen, below)
                const uint32_t use = base + v_at(g, j);
                if (!wait_on(M, M.full[use % Sh::kSlots], use / Sh::kSlots & 1, P)) return leave();
                char *v = smem + Sh::kRing + use % Sh::kSlots * Sh::kTileBytes;
                const int r0 = max(0, -shift), gone = g.s.T - shift;
                for (int i = tid & 255; i < (kTile - r0) * (D / 8); i += 256) {
                    const int r = r0 + i / (D / 8), c = i % (D / 8);
                    uint4 *at = reinterpret_cast<uint4 *>(v + (c >> 3) * Sh::kPanel + r * 128 +
                                                          ((c & 7) << 4));
                    if (r >= gone) {
                        *at = make_uint4(0, 0, 0, 0);
                    } else {
                        uint4 x = *at;
                        const uint32_t a = nonfinite_bits<FP16>(x.x), b = nonfinite_bits<FP16>(x.y),
                                       c4 = nonfinite_bits<FP16>(x.z),
                                       d4 = nonfinite_bits<FP16>(x.w);
                        if (a | b | c4 | d4) {
                            *at = make_uint4(x.x & ~a, x.y & ~b, x.z & ~c4, x.w & ~d4);
                            const int i = r + shift;
                            atomicOr(&sc.nonfinite[i >> 5], 1u << (i & 31));
                        }
                    }
                }
                fence_async_smem();
            }
            // P's first half of the slots is complete when both warps of a row have
            // done theirs of it, and its products start under the second half
            const auto done = [&](int part) {
                tc_fence_before();
                __syncwarp();  // a warp's one arrival: 256 on one barrier take their time
                if (lane == 0) mbar_arrive(smem_u32(&M.p_full[w][part]));
            };
            if (warp_on) {
                uint32_t s[H];  // columns 32 h and up of each half of S
                tmem_ld32(ts + 32 * h, s);
                tmem_ld32(ts + H + 32 * h, s + 32);
                tmem_wait_ld();
                if (tail_tile) {
                    uint32_t up[kMaskWords] = {};  // the node's ancestors and itself
                    for (int i = node; i >= 0; i = sc.parent[i])
#pragma unroll
                        for (int q = 0; q < kMaskWords; ++q)
                            if (i >> 5 == q) up[q] |= 1u << (i & 31);
                    const auto word = [&](int i) -> uint32_t {
                        uint32_t x = i < 0 ? 0xffffffffu : 0u;
#pragma unroll
                        for (int q = 0; q < kMaskWords; ++q)
                            if (i == q) x = up[q];
                        return x;
                    };
#pragma unroll
                    for (int q = 0; q < H / 32; ++q) {
                        const int at = H * q + 32 * h + shift;
                        const uint32_t see =
                            __funnelshift_r(word(at >> 5), word((at >> 5) + 1), at & 31);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(see >> c & 1)) s[32 * q + c] = __float_as_uint(ninf);
                    }
                }
                float m4[4] = {ninf, ninf, ninf, ninf};
#pragma unroll
                for (int i = 0; i < H; i += 8)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        m4[c] = fmaxf(m4[c], fmaxf(__uint_as_float(s[i + c]), __uint_as_float(s[i + c + 4])));
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c2;
                // Both warps have read S when the barrier opens: P may go over it.
                if (pair_any(pair_bar, mine && mx > m_ref + Range<FP16>::kSlack)) {
                    M.x[2 * w + h][row] = mx;
                    pair_any(pair_bar, false);
                    const float top = fmaxf(m_ref, fmaxf(M.x[2 * w][row], M.x[2 * w + 1][row]));
                    const float f = m_ref == top ? 1.0f : ex2_approx(m_ref - top);
                    m_ref = top;
                    l *= f;
                    if (!fresh) {
#pragma unroll 1
                        for (int c = h * (D / 2); c < (h + 1) * (D / 2); c += 16) {
                            uint32_t o[16];
                            const uint32_t at = tmem + lanes + Sh::kO + w * D + c;
                            tmem_ld16(at, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(at, o);
                        }
                    }
                }
                const float off = Range<FP16>::kShift - (m_ref == ninf ? 0.0f : m_ref);
                const f32x2 c22 = pack2(c2, c2), off2 = pack2(off, off);
                f32x2 sum0 = pack2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int c = 32 * q + 2 * i;
                        const float2 x = unpack2(fma2(
                            pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), c22, off2));
                        const float a = ex2_approx(x.x), b = ex2_approx(x.y);
                        if (i & 1)
                            sum1 = add2(sum1, pack2(a, b));
                        else
                            sum0 = add2(sum0, pack2(a, b));
                        p[i] = pack_half<FP16>(a, b);
                    }
                    tmem_st16(ts + 32 * q + 16 * h, p);
                    tmem_wait_st();
                    done(q);
                }
                const float2 sum = unpack2(add2(sum0, sum1));
                l += sum.x + sum.y;
            } else {
                done(0);
                done(1);
            }
            fresh = false;
        }
        // the item's sums
        const bool used1 = pair || n > 1;
        if ((!pair || w == 0) && !wait_on(M, M.o_full[0], o_phase & 1, P)) return leave();
        if (used1 && (!pair || w == 1) && !wait_on(M, M.o_full[1], o_phase >> 1, P))
            return leave();
        o_phase ^= used1 ? 3 : 1;
        tc_fence_after();
        base += 2 * n;
        float wgt[2] = {1.0f, 1.0f};
        float mf = m_ref, lf = l;
        if (!pair) {
            // join the groups, each of the four warpgroups a quarter of the columns
            M.x[2 * w][row] = m_ref;  // both halves' is the same
            soft_sync();
            const float m0 = M.x[0][row], m1 = M.x[2][row];
            mf = fmaxf(m0, m1);
            wgt[0] = m0 == ninf ? 0.0f : fmaxf(ex2_approx(m0 - mf), kTiny);
            wgt[1] = m1 == ninf ? 0.0f : fmaxf(ex2_approx(m1 - mf), kTiny);
            soft_sync();
            M.x[2 * w + h][row] = l * wgt[w];
            soft_sync();
            lf = M.x[0][row] + M.x[1][row];
            if (used1) lf += M.x[2][row] + M.x[3][row];
        } else {
            M.x[2 * w + h][row] = l;
            soft_sync();  // of all: group 0's sc.nonfinite, too
            lf = M.x[2 * w][row] + M.x[2 * w + 1][row];
        }
        if (sc.bad) lf = NAN;
        if (warp_on) {
            const bool whole = g.first && g.last;
            const float inv = whole ? (lf == 0.0f ? 0.0f : 1.0f / lf) : 1.0f;
            const int64_t orow = g.s.row0 + node;
            const int c_begin = pair ? h * (D / 2) : (2 * w + h) * CW;
            const int c_end = c_begin + (pair ? D / 2 : CW);
            const int piece = g.first ? 1 : 0;  // a CTA's first and last segments may be pieces
            const int64_t at = ((int64_t)blockIdx.x * 2 + piece) * (2 * kTile) + r_item;
            bool any_odd = false;
#pragma unroll
            for (int q = 0; q < kMaskWords; ++q) any_odd |= sc.nonfinite[q] != 0;
#pragma unroll 1
            for (int c = c_begin; c < c_end; c += CW) {
                uint32_t o[CW];
                float f[CW];
                tmem_ld_n<CW>(tmem + lanes + Sh::kO + (pair ? w * D : 0) + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < CW; ++i) f[i] = __uint_as_float(o[i]) * wgt[0];
                if (!pair && used1) {
                    tmem_ld_n<CW>(tmem + lanes + Sh::kO + D + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < CW; ++i) f[i] = fmaf(__uint_as_float(o[i]), wgt[1], f[i]);
                }
                if (any_odd && mine && !sc.bad) {
                    // a seen inf or NaN decides its element whatever its weight (a bad
                    // segment has no page to read: its sum is NaN already)
                    for (int j = node; j >= 0; j = sc.parent[j]) {
                        if (!(sc.nonfinite[j >> 5] >> (j & 31) & 1)) continue;
                        const int s = g.s.L + j;
                        const uint32_t *v = reinterpret_cast<const uint32_t *>(
                            P.c.v + (int64_t)g.head * P.c.hs + page_of(P.c, g.b, s) * P.c.ps +
                            (int64_t)place_of(P.c, s).token * P.c.ts + c * 2);
#pragma unroll
                        for (int i = 0; i < CW / 2; ++i) {
                            const uint32_t x = v[i], bits = nonfinite_bits<FP16>(x);
                            if (bits & 0xffffu) f[2 * i] += half_at<FP16>(x, 0);
                            if (bits >> 16) f[2 * i + 1] += half_at<FP16>(x, 1);
                        }
                    }
                }
                if (mine) {
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(P.out + orow * P.o_rs +
                                                               (int64_t)qh * P.o_hs + c * 2);
#pragma unroll
                        for (int i = 0; i < CW / 8; ++i)
                            dst[i] = make_uint4(
                                pack_half<FP16>(f[8 * i] * inv, f[8 * i + 1] * inv),
                                pack_half<FP16>(f[8 * i + 2] * inv, f[8 * i + 3] * inv),
                                pack_half<FP16>(f[8 * i + 4] * inv, f[8 * i + 5] * inv),
                                pack_half<FP16>(f[8 * i + 6] * inv, f[8 * i + 7] * inv));
                    } else {
#pragma unroll
                        for (int i = 0; i < CW / 8; ++i)
                            st_global_8(P.piece_o + at * D + c + 8 * i, f + 8 * i);
                    }
                }
            }
            if (mine && h == 0 && (pair || w == 0)) {
                if (!whole)
                    P.piece_ml[at] = make_float2(mf, lf);
                else if (P.lse)
                    P.lse[orow * P.heads + qh] =
                        (mf + log2f(lf) - Range<FP16>::kShift) * 0.6931471805599453f;
            }
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&M.seg_empty[seg & 1]));
    }
}

// ---------------------------------------------------------------------------
// scouts: Q tiles, pages and parents, a segment ahead

template <bool FP16, int D>
__device__ void scout_role(const TreeAttnParams &P, Misc &M, char *smem, Walk walk) {
    using Sh = Shape<D>;
    constexpr int C = D / 8;  // 16-byte chunks of a row
    const int tid = threadIdx.x - (kAttnThreads - kScoutThreads);
    const uint32_t q = smem_u32(smem);
    uint32_t seg = 0, uses[2] = {0, 0}, turn = 0;
    Segment g;
    for (;; ++seg) {
        if (!walk.next(P, g)) {
            if (wait_on(M, M.seg_empty[seg & 1], (seg >> 1 & 1) ^ 1, P)) {
                if (tid == 0) M.seg[seg & 1].g.n = 0;
                mbar_arrive(smem_u32(&M.seg_full[seg & 1]));
            }
            break;
        }
        bool ok = true;
        // the checks' first loads go out before the copies
        const int t_begin = g.tile0 * kTile, t_end = min((g.tile0 + g.n) * kTile, g.s.L + g.s.T);
        const bool tail = t_end > g.s.L;
        const int pg0 = place_of(P.c, t_begin).index, pg1 = place_of(P.c, t_end - 1).index;
        const bool page_ok = pg0 + tid > pg1 || page_at(P.c, g.b, pg0 + tid) >= 0;
        int up[kMaxNodes / kScoutThreads];
#pragma unroll
        for (int i = 0; i < kMaxNodes / kScoutThreads; ++i) {
            const int j = tid + i * kScoutThreads;
            up[i] = tail && j < g.s.T ? P.t.parent[(int64_t)g.b * P.t.max_nodes + j] : -1;
        }
        // Q rows into their tiles, 16-byte chunks swizzled within 8 rows
        for (int i = 0; i < (g.pair ? 2 : 1); ++i) {
            const int x = g.pair ? i : turn;
            ok = ok && wait_on(M, M.q_empty[x], (uses[x]++ & 1) ^ 1, P);
            if (!ok) break;
            const int r_first = i * kTile, r_count = min(kTile, g.rows - r_first);
            constexpr int R = kScoutThreads / C;  // rows at a time
            const int c = tid % C, dn = R / P.G, dh = R - dn * P.G;
            const int gr = g.block * 2 * kTile + r_first + tid / C;
            int node = gr / P.G, hh = gr - node * P.G;
            const uint32_t tile = q + x * Sh::kTileBytes + (c >> 3) * Sh::kPanel;
            const char *src = P.q + g.s.row0 * P.q_rs + (int64_t)g.head * P.G * P.q_hs + c * 16;
            for (int r = tid / C; r < r_count; r += R) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 tile + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                             "l"(src + node * P.q_rs + hh * P.q_hs)
                             : "memory");
                node += dn;
                hh += dh;
                if (hh >= P.G) {
                    hh -= P.G;
                    ++node;
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            mbar_arrive(smem_u32(&M.q_full[x]));
            if (seg == 0 && i == 0) mbar_arrive(smem_u32(&M.begun));
        }
        if (!g.pair) turn ^= 1;
        // pages and parents
        ok = ok && wait_on(M, M.seg_empty[seg & 1], (seg >> 1 & 1) ^ 1, P);
        if (!scouts_all(ok)) break;
        Scouted &sc = M.seg[seg & 1];
        int bad = page_ok ? 0 : SPECVERIFY_STATUS_BAD_CACHE;
        for (int i = pg0 + tid + kScoutThreads; i <= pg1; i += kScoutThreads)
            if (page_at(P.c, g.b, i) < 0) bad |= SPECVERIFY_STATUS_BAD_CACHE;
        if (tail)
#pragma unroll
            for (int i = 0; i < kMaxNodes / kScoutThreads; ++i) {
                const int j = tid + i * kScoutThreads;
                if (j >= g.s.T) continue;
                const bool no = j == 0 ? up[i] != -1 : (up[i] < 0 || up[i] >= j);
                sc.parent[j] = (int8_t)(no ? -1 : up[i]);
                if (no) bad |= SPECVERIFY_STATUS_BAD_TREE;
            }
        if (tid < kMaskWords) sc.nonfinite[tid] = 0;
        if (tid == 0) {
            sc.g = g;
            sc.bad = 0;
        }
        scouts_all(true);
        if (bad) {
            atomicOr(P.status, bad);
            sc.bad = 1;
        }
        mbar_arrive(smem_u32(&M.seg_full[seg & 1]));
    }
}

// ---------------------------------------------------------------------------
// products

template <bool FP16, int D>
__device__ void mma_role(const TreeAttnParams &P, Misc &M, char *smem, Walk walk, uint32_t tmem) {
    using Sh = Shape<D>;
    constexpr uint32_t dqk = mma_desc(FP16, false, kTile, kTile), dpv = mma_desc(FP16, true, kTile, D);
    const uint32_t q0 = smem_u32(smem), ring = q0 + Sh::kRing;
    const bool on = elect_one();
    uint32_t base = 0, uses[2] = {0, 0}, turn = 0, p_phase[2] = {0, 0};
    Segment g;
    bool ok = true;
    while (ok && walk.next(P, g)) {
        const int steps = g.pair ? 2 * g.n : g.n;
        // step t: group t % 2, tile t (or t / 2 when both groups take every tile)
        uint32_t slot_k = 0, phase_k = 0;  // of the next step's K, found while P is waited for
        const auto find_k = [&](int t) {
            const uint32_t use = base + k_at(g, g.pair ? t >> 1 : t);
            slot_k = use % Sh::kSlots;
            phase_k = use / Sh::kSlots & 1;
        };
        const auto qk = [&](int t) {
            const int w = t & 1;
            const uint32_t slot = slot_k;
            const int x = g.pair ? w : turn;
            if (t == 0 || (g.pair && t == 1)) ok = wait_on(M, M.q_full[x], uses[x]++ & 1, P);
            if (!g.pair || w == 0) ok = ok && wait_on(M, M.full[slot], phase_k, P);
            if (!ok) return;
            tc_fence_after();
            const uint32_t a = q0 + x * Sh::kTileBytes, b = ring + slot * Sh::kTileBytes;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k >> 2) * Sh::kPanel + (k & 3) * 32;
                mma_ss(tmem + Sh::kS + w * kTile, smem_desc(a + off, 0), smem_desc(b + off, 0), dqk,
                       k > 0, on);
            }
            mma_commit(smem_u32(&M.s_full[w]), on);
            if (g.pair ? t + 2 >= steps : t + 1 == steps) mma_commit(smem_u32(&M.q_empty[x]), on);
            if (!g.pair || w == 1) mma_commit(smem_u32(&M.empty[slot]), on);
        };
        find_k(0);
        if (ok) qk(0);
        find_k(1);
        if (ok && steps > 1) qk(1);
        for (int t = 0; ok && t < steps; ++t) {
            const int j = g.pair ? t >> 1 : t, w = t & 1;
            const uint32_t use = base + v_at(g, j), slot = use % Sh::kSlots;
            find_k(t + 2);
            if (!g.pair || w == 0) ok = wait_on(M, M.full[slot], use / Sh::kSlots & 1, P);
            const uint32_t b = ring + slot * Sh::kTileBytes;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                ok = ok && wait_on(M, M.p_full[w][part], p_phase[w], P);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = part * kTile / 32; k < (part + 1) * kTile / 32; ++k)
                    mma_ts(tmem + Sh::kO + w * D, tmem + Sh::kS + w * kTile + k * 8,
                           smem_desc(b + k * 2048, Sh::kPanel), dpv, t >= 2 || k > 0, on);
            }
            p_phase[w] ^= 1;
            if (!ok) break;
            if (!g.pair || w == 1) mma_commit(smem_u32(&M.empty[slot]), on);
            if (t + 2 >= steps) mma_commit(smem_u32(&M.o_full[w]), on);
            if (t + 2 < steps) qk(t + 2);
        }
        base += 2 * g.n;
        if (!g.pair) turn ^= 1;
    }
    // No product, nor the arrival of one, outlives the CTA. Whoever reads the last ones
    // may have given up waiting for them, also where every wait of this warp was met.
    mma_commit(smem_u32(&M.drain), on);
    mbar_wait_bounded(smem_u32(&M.drain), 0);
}

// ---------------------------------------------------------------------------
// copies

template <int D>
__device__ void load_role(const TreeAttnParams &P, const CUtensorMap *mk, const CUtensorMap *mv,
                          Misc &M, char *smem, Walk walk) {
    using Sh = Shape<D>;
    const int lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(smem) + Sh::kRing;
    const int box = P.box;
    uint32_t use = 0;
    Segment g;
    bool ok = true;
    while (ok && walk.next(P, g)) {
        const int len = g.s.L + g.s.T;
        const auto page_id = [&](int j) -> int {  // of the lane's box in tile j, -1: none
            const int s = (g.tile0 + j) * kTile + lane * box;
            return j < g.n && lane * box < kTile && s < len ? (int)page_of(P.c, g.b, s) : -1;
        };
        const auto copy = [&](const CUtensorMap *map, int j, int page) {
            const uint32_t slot = use % Sh::kSlots, bar = smem_u32(&M.full[slot]);
            ok = wait_on(M, M.empty[slot], (use / Sh::kSlots & 1) ^ 1, P);
            // the first queries come ahead of a ring's worth of keys, which would
            // keep them in the memory's queue for microseconds
            if (use == 2) ok = ok && wait_on(M, M.begun, 0, P);
            if (!ok) return;
            ++use;
            const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, page >= 0));
            if (lane == 0) mbar_arrive_expect_tx(bar, boxes * box * D * 2);
            __syncwarp();
            if (page >= 0) {
                const int s = (g.tile0 + j) * kTile + lane * box;
                const uint32_t dst = ring + slot * Sh::kTileBytes + lane * box * 128;
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tile_load(dst + c * Sh::kPanel, map, c * 64, place_of(P.c, s).token, g.head, page, bar);
            }
            __syncwarp();
        };
        // the order of k_at and v_at; page ids are fetched a tile ahead
        int now = page_id(0), next = page_id(1);
        copy(mk, 0, now);
        for (int j = 0; ok && j < g.n; ++j) {
            const int after = page_id(j + 2);
            if (!g.pair && j + 1 < g.n) copy(mk, j + 1, next);
            if (ok) copy(mv, j, now);
            if (ok && g.pair && j + 1 < g.n) copy(mk, j + 1, next);
            now = next;
            next = after;
        }
    }
    // no copy outlives the CTA
    for (uint32_t u = use > Sh::kSlots ? use - Sh::kSlots : 0; u < use; ++u)
        mbar_wait_bounded(smem_u32(&M.full[u % Sh::kSlots]), u / Sh::kSlots & 1);
}

// ---------------------------------------------------------------------------

template <bool FP16, int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
    tree_attn_kernel(const __grid_constant__ TreeAttnParams P,
                     const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
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
            mbar_init(smem_u32(&M.q_empty[w]), 1);
            mbar_init(smem_u32(&M.seg_full[w]), kScoutThreads);
            mbar_init(smem_u32(&M.seg_empty[w]), kSoftThreads);
            mbar_init(smem_u32(&M.s_full[w]), 1);
            mbar_init(smem_u32(&M.p_full[w][0]), kSoftThreads / 64);
            mbar_init(smem_u32(&M.p_full[w][1]), kSoftThreads / 64);
            mbar_init(smem_u32(&M.o_full[w]), 1);
        }
        mbar_init(smem_u32(&M.begun), kScoutThreads);
        mbar_init(smem_u32(&M.drain), 1);
        M.abort = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) tmem_alloc(smem_u32(&M.tmem), kTmemCols);
    after_previous();

    // the line: each thread a run of sequences, a scan over the threads
    const int per = (P.t.B + kAttnThreads - 1) / kAttnThreads;
    const int b0 = min(P.t.B, tid * per), b1 = min(P.t.B, b0 + per);
    long long first = 0, all = 0;  // units of the run: the first block of rows, every block
    for (int b = b0; b < b1; ++b) {
        const Seq s = seq_of(P, b);
        first += s.units(P, 0);
        all += (long long)s.units(P, 0) * s.blocks;
        if (s.tiles == 0 && s.T != 0 && b % (int)gridDim.x == (int)blockIdx.x) {
            // a bad sequence: NaN in the rows that it names, if it names rows
            const int bad = seq_error(P, s.T, s.row0, s.L);
            atomicOr(P.status, bad);
            if (bad == SPECVERIFY_STATUS_BAD_CACHE)
                for (int64_t r = s.row0; r < s.row0 + s.T; ++r)
                    for (int h = 0; h < P.heads; ++h) {
                        for (int c = 0; c < D; ++c)
                            reinterpret_cast<uint16_t *>(P.out + r * P.o_rs + h * P.o_hs)[c] = 0x7FFF;
                        if (P.lse) P.lse[r * P.heads + h] = NAN;
                    }
        }
    }
    // units before this thread's, and everybody's
    const auto scan = [&](long long mine, long long &sum) {
        long long incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) M.scan[warp] = incl;
        __syncthreads();
        long long before = incl - mine;
        sum = 0;
        for (int i = 0; i < kAttnThreads / 32; ++i) {
            if (i < warp) before += M.scan[i];
            sum += M.scan[i];
        }
        return before;
    };
    tc_fence_before();
    long long total, in_block = 0;
    long long before = scan(all, total);
    tc_fence_after();
    const Cut cut(total, gridDim.x);
    const int cta = min((int)blockIdx.x, cut.ctas);
    const long long lo = cut.at(cta), hi = cut.at(min(cta + 1, cut.ctas));
    long long start = 0;  // of the block on the line
    for (int block = 0; block < P.blocks; ++block) {
        long long mine = first;
        if (P.blocks > 1) {
            __syncthreads();
            mine = 0;
            for (int b = b0; b < b1; ++b) mine += seq_of(P, b).units(P, block);
            before = scan(mine, in_block);
        }
        if (lo < hi && start + before <= lo && lo < start + before + mine) {
            long long at = start + before;
            for (int b = b0; b < b1; ++b) {
                const int n = seq_of(P, b).units(P, block);
                if (lo < at + n) {
                    M.b0 = b;
                    M.block0 = block;
                    M.rest0 = (int)(lo - at);
                    break;
                }
                at += n;
            }
        }
        start += in_block;
        if (lo < start) break;
    }
    __syncthreads();
    Walk walk{M.b0, M.block0, M.rest0, hi - lo};
    const uint32_t tmem = M.tmem;
    if (warp < kSoftThreads / 32) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        softmax_role<FP16, D>(P, M, smem, tmem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    }
    if (warp == kMmaWarp) {
        mma_role<FP16, D>(P, M, smem, walk, tmem);
    } else if (warp > kLoadWarp) {
        scout_role<FP16, D>(P, M, smem, walk);
    } else if (warp == kLoadWarp) {
        load_role<D>(P, &mk, &mv, M, smem, walk);
        // the item that this CTA begins and does not end, for the joining kernel
        if (lane == 0) {
            AttnOwner o{};
            Walk v = walk;
            Segment g;
            while (v.next(P, g)) {
                if (g.first && !g.last) {  // the CTA's last segment: the line goes on at hi
                    o.pieces = cut.of(hi + g.s.tiles - g.n - 1) - (int)blockIdx.x + 1;
                    o.rows = g.rows;
                    o.first_row = g.block * 2 * kTile;
                    o.head = g.head;
                    o.row0 = g.s.row0;
                }
            }
            P.owner[blockIdx.x] = o;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_free(tmem, kTmemCols);
}

// Joins the pieces of the items that were cut: block (c, y) rows 8 y and up of
// the item that CTA c began, two a warp. Piece 0 is c's last segment, the next
// CTAs' first segments follow. Bound by the latency of its loads: the first
// kAhead pieces are read before anything is known of their weights.
constexpr int kJoinWarps = 4, kJoinRows = 2;

template <bool FP16, int D, int kAhead>
__global__ void __launch_bounds__(kJoinWarps * 32, kAhead <= 3 ? 8 : 4) tree_join_kernel(const __grid_constant__ TreeAttnParams P) {
    after_previous();
    constexpr int W = D / 32;
    using Vec = typename std::conditional<W == 4, float4, float2>::type;
    const AttnOwner o = P.owner[blockIdx.x];
    const int lane = threadIdx.x & 31;
    const int r0 = (blockIdx.y * kJoinWarps + (threadIdx.x >> 5)) * kJoinRows;
    if (o.pieces == 0 || r0 >= o.rows) return;
    const auto at = [&](int i, int k) -> int64_t {  // rows past the item's are in its slot too
        return ((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * (2 * kTile) + r0 + k;
    };
    const auto piece = [&](int i, int k, float *x) {
        *reinterpret_cast<Vec *>(x) = *reinterpret_cast<const Vec *>(P.piece_o + at(i, k) * D + lane * W);
    };
    float x[kAhead][kJoinRows][W], m[kJoinRows], l[kJoinRows] = {}, f[kJoinRows][W] = {};
    float2 ml[kAhead][kJoinRows];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (i < o.pieces)
#pragma unroll
            for (int k = 0; k < kJoinRows; ++k) {
                ml[i][k] = P.piece_ml[at(i, k)];
                piece(i, k, x[i][k]);
            }
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
        m[k] = -INFINITY;
        for (int i = lane; i < o.pieces; i += 32) m[k] = fmaxf(m[k], P.piece_ml[at(i, k)].x);
    }
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k)
        for (int s = 16; s > 0; s >>= 1) m[k] = fmaxf(m[k], __shfl_xor_sync(0xffffffffu, m[k], s));
    const auto add = [&](int k, float2 a, const float *v) {
        const float wgt = a.x == -INFINITY ? 0.0f : fmaxf(ex2_approx(a.x - m[k]), kTiny);
        l[k] = fmaf(a.y, a.x == -INFINITY ? 1.0f : wgt, l[k]);  // a NaN sum stays one
#pragma unroll
        for (int c = 0; c < W; ++c) f[k][c] = fmaf(v[c], wgt, f[k][c]);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (i < o.pieces)
#pragma unroll
            for (int k = 0; k < kJoinRows; ++k) add(k, ml[i][k], x[i][k]);
    for (int i0 = kAhead; i0 < o.pieces; i0 += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i < o.pieces)
#pragma unroll
                for (int k = 0; k < kJoinRows; ++k) {
                    ml[i][k] = P.piece_ml[at(i0 + i, k)];
                    piece(i0 + i, k, x[i][k]);
                }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i < o.pieces)
#pragma unroll
                for (int k = 0; k < kJoinRows; ++k) add(k, ml[i][k], x[i][k]);
    }
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
        if (r0 + k >= o.rows) break;
        const int gr = o.first_row + r0 + k, node = gr / P.G, h = o.head * P.G + gr - node * P.G;
        const int64_t row = o.row0 + node;
        const float inv = l[k] == 0.0f ? 0.0f : 1.0f / l[k];
        uint32_t *dst = reinterpret_cast<uint32_t *>(P.out + row * P.o_rs + (int64_t)h * P.o_hs) +
                        lane * (W / 2);
#pragma unroll
        for (int c = 0; c < W / 2; ++c)
            dst[c] = pack_half<FP16>(f[k][2 * c] * inv, f[k][2 * c + 1] * inv);
        if (P.lse && lane == 0)
            P.lse[row * P.heads + h] = (m[k] + log2f(l[k]) - Range<FP16>::kShift) * 0.6931471805599453f;
    }
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn g_encode = nullptr;

template <bool FP16, int D>
cudaError_t launch(const TreeAttnParams &p, const CUtensorMap &mk, const CUtensorMap &mv, int ctas,
                   cudaStream_t s) {
    const cudaError_t e = launch_after(tree_attn_kernel<FP16, D>, dim3((unsigned)ctas), kAttnThreads,
                                       Shape<D>::kSmem, s, 1, p, mk, mv);
    if (e != cudaSuccess) return e;
    const int64_t most = std::min((int64_t)2 * kTile, (int64_t)p.t.max_nodes * p.G);
    const unsigned y = (unsigned)((most + kJoinWarps * kJoinRows - 1) / (kJoinWarps * kJoinRows));
    const dim3 grid((unsigned)ctas, y);
    // With an item for every second CTA, cut items have two or three pieces (and
    // there are many: fewer registers, more rows at once); with few items, more.
    if ((int64_t)p.t.B * p.c.kv_heads * 2 >= ctas)
        return launch_after(tree_join_kernel<FP16, D, 3>, grid, kJoinWarps * 32, 0, s, 1, p);
    return launch_after(tree_join_kernel<FP16, D, 8>, grid, kJoinWarps * 32, 0, s, 1, p);
}

template <bool FP16, int D>
cudaError_t prepare() {
    return cudaFuncSetAttribute(tree_attn_kernel<FP16, D>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem);
}

}  // namespace

bool cache_map(const CacheParams &c, const char *base, int box, CUtensorMap *map) {
    const cuuint64_t dim[4] = {(cuuint64_t)c.d, (cuuint64_t)c.page, (cuuint64_t)c.kv_heads,
                               (cuuint64_t)c.num_pages};
    // the stride of a dimension of one is never used, but has to be a legal one
    const cuuint64_t stride[3] = {(cuuint64_t)c.ts, (cuuint64_t)(c.kv_heads > 1 ? c.hs : c.ts),
                                  (cuuint64_t)(c.num_pages > 1 ? c.ps : c.ts)};
    const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1}, one[4] = {1, 1, 1, 1};
    return g_encode(map,
                    c.fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                    const_cast<char *>(base), dim, stride, boxes, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int cache_box(int page) {
    int box = kTile;
    while (page % box != 0) box /= 2;
    return box;
}

size_t attn_workspace(int ctas) {
    return (size_t)ctas * 2 * 2 * kTile * (128 * sizeof(float) + sizeof(float2)) +
           (size_t)ctas * sizeof(AttnOwner);
}

void attn_place(TreeAttnParams &p, void *ws, int ctas) {
    const int64_t rows = (int64_t)ctas * 2 * 2 * kTile;
    p.piece_o = static_cast<float *>(ws);
    p.piece_ml = reinterpret_cast<float2 *>(p.piece_o + rows * 128);
    p.owner = reinterpret_cast<AttnOwner *>(p.piece_ml + rows);
}

cudaError_t prepare_tree() {
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                               cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
        g_encode = reinterpret_cast<EncodeFn>(fn);
    }
    cudaError_t e = prepare<false, 64>();
    if (e == cudaSuccess) e = prepare<false, 128>();
    if (e == cudaSuccess) e = prepare<true, 64>();
    if (e == cudaSuccess) e = prepare<true, 128>();
    return e;
}

cudaError_t launch_tree_attention(TreeAttnParams p, int num_sms, cudaStream_t s) {
    CUtensorMap mk, mv;
    p.box = cache_box(p.c.page);
    p.blocks = (int32_t)(((int64_t)p.t.max_nodes * p.G + 2 * kTile - 1) / (2 * kTile));
    if (!cache_map(p.c, p.c.k, p.box, &mk) || !cache_map(p.c, p.c.v, p.box, &mv))
        return cudaErrorInvalidValue;
    if (p.c.fp16)
        return p.c.d == 128 ? launch<true, 128>(p, mk, mv, num_sms, s)
                            : launch<true, 64>(p, mk, mv, num_sms, s);
    return p.c.d == 128 ? launch<false, 128>(p, mk, mv, num_sms, s)
                        : launch<false, 64>(p, mk, mv, num_sms, s);
}

}  // namespace sv
