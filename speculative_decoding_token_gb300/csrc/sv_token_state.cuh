// sv_token_state.cuh -- what the warps of the token log-probability and
// distillation kernel (sv_token.cuh) share: its sizes, a CTA's state, partial sums,
// waits, and the words that a cluster's CTAs send one another.
#pragma once

#include "sv_token_math.cuh"

namespace sv {

namespace token {

constexpr int kConsumers = 8;                     // warps
constexpr int kScout = kConsumers, kProducer = kScout + 1, kBeside = kProducer + 1, kEpilogue = kBeside + 1;  // (beside: patcher or top tokens)
constexpr int kThreads = (kEpilogue + 1) * 32;
constexpr int kTeam = kConsumers * 32;            // a thread takes every kTeam-th 16-byte vector of a chunk
constexpr int kMaxSlots = 26;
constexpr int kDepth = 4;                         // rows between the scout and the epilogue at most
constexpr int kTopDepth = 2;                      // the same where top tokens are asked for (their buffers are large)
// Chunks that a row has left to copy when the next is asked for: 2 to 5 us pass until that one's first copy. Gradients of
// 512 rows of 256000 fp32 logits: 197 us for none, 184 for two; rows of 152064 bf16: 200, 199 and, for five, 206 (the sooner a
// row is taken the worse the rows are balanced).
constexpr int kLead = 2;
constexpr int kMaxCluster = 16;
// Groups of a thread's vectors in a slice whose maxima are kept: as many as shared memory has room for (two rows of 24 x 256
// halves) beside four slots of the ring and the words of the largest cluster. A group is 2^n chunks, the least that a slice fits
// in: one up to 196608 bf16 or 98304 fp32 logits. (Larger groups have more vectors read again: of 2000 rows of 152064 with 64 top
// tokens, 132 us for groups of two chunks, 124.9 for one.)
constexpr int kGroupRows = 24;
constexpr int kMine = 256, kKept = 512;           // groups that may hold top tokens, a warp's and all
constexpr unsigned kLost = 1u << 24;
constexpr int kKeys = 512;                        // tokens among them
// Where top tokens are asked for, a cluster's slices have this many vectors at least, and its CTAs send its first this many keys
// at most: that one has to put them in order too (in a graph, us for clusters of 1, 2, 4, 8, 16: a row of 152064 bf16 logits and
// k = 5: 13.9, 11.0, 8.7, 8.6, 10.4; five of 128256, k = 20: 13.4, 11.1, 10.5, 14.0, 24; twelve of 152064, k = 64: 16.0, 17.4, 21;
// 20 of 32000, k = 20: 8.1, 10.0, 12.7).
constexpr int kLeastTop = 4096, kGathered = 64;
constexpr int kHash = 1024;

enum State { kLive = 0, kSkip = 1, kBad = 2, kEnd = 3 };

// What a kernel is compiled for.
template <int kDtype, bool kIsList, bool kIsGrad, bool kHasEntropy, bool kHasTop, bool kHasRank>
struct Kind {
    static constexpr int DT = kDtype;
    static constexpr bool List = kIsList, Grad = kIsGrad, Ent = kHasEntropy, Top = kHasTop, Rank = kHasRank;
    static constexpr int kSize = DT == SV_DT_FP32 ? 4 : 2;
    static constexpr int kPer = 16 / kSize;  // logits of a vector
    static constexpr uint32_t kNegInf = DT == SV_DT_FP32 ? 0xff800000u : 0xff80ff80u;
    static constexpr int kVecs = 4;  // of a chunk, a thread
    static constexpr int kId = DT + 2 * (List ? 7 + Grad : Grad ? 5 + Ent : Rank ? 3 + Top : Top ? 2 : Ent);  // in TokenRooms
    // numbers of a Part that a cluster's CTAs send one another
    static constexpr int kWords = 2 + (Ent ? 1 : 0) + (Rank ? 1 : 0);
    static constexpr int kChunkVecs = kTeam * kVecs, kChunkBytes = kChunkVecs * 16;
};

// What the scout knows of a row.
struct Row {
    const char *z;
    long long entry;
    int state;
    int y;
    int bad;       // what was found wrong with its list
    float zy;
    // of a list: what it leaves of one, the logarithm, and what all of p is more than one
    float p_rest, p_rest_l, rest_h, rest_l, over;
    // the draft's largest logit z of it and (RKL) its p and ln p, the sum of e^((z_k - z) / T), and (RKL) of that times (z_k - z) / T -
    // (ln p_k - ln p)
    float zmax, p0, p0_l, lp0, zsum, zsum_l, cross;
    float p0_inv, rest_inv;  // (RKL) 1 / p of it and 1 / p of the rest, no less than 2^-20
    float tmax, t_h, t_l;  // the target's largest logit, and the logarithm of the sum relative to it
    float g, h;    // what the gradient is multiplied by
};

// Sums over part of a row: s of 2^x and t of 2^x x, x = z c - R, or (z - m) c (see plain), m a logit near the largest (-inf where
// there is none but -inf); n tokens before the given one, -1: a bad logit.
struct Part {
    float m, s, t;
    int n;
};

struct Shared {
    uint64_t full[kMaxSlots], ready[kMaxSlots], empty[kMaxSlots];
    // of a row: known; done with; all known of its entry; its copies issued; the CTA's sums there, its bounds (top
    // tokens); of a gradient: what the second reading needs, all stored
    uint64_t row_full[kDepth], row_free[kDepth], scouted[kDepth], sent[kDepth], summed[kDepth], bounded[kDepth], known[kDepth], stored[kDepth];
    uint64_t gathered, granted, acked;
    uint4 grant;          // the answer to a request for another row
    Row row[kDepth];
    Part part[kDepth][kConsumers];  // of the CTA's warps where a row is one CTA's
    float4 coef[kDepth];  // of the gradient: m, a, b (see store_slice)
    float fix[kDepth];    // the given token's gradient (a list's tokens': Lists::lp)
    int good[kDepth];
    int asked;            // requests made (the first CTA's)
    int32_t abort;
};

// Top tokens: a key is a logit's bits, made to order as it does, over its
// token's, inverted: keys fall in the order of alternatives, and 0 is none.
struct SharedTop {
    uint16_t most[kTopDepth][kGroupRows][kTeam];  // the groups' maxima, upper halves of their bits
    uint32_t bound[kTopDepth][kConsumers];        // the order bits of a number that enough of the warp's tokens reach
    uint16_t mine[kConsumers][kMine];             // groups of a warp's share that may hold top tokens
    uint16_t kept[kKept];                         // and of all of them, where that was not enough
    alignas(16) unsigned long long keys[kTopDepth][kKeys];
    alignas(16) unsigned long long gathered[kGathered];
    unsigned long long best[kMaxAlternatives];    // the first k of a row, in order
    unsigned found[kTopDepth];                    // keys; kLost and more: not all of them
};

// Lists of kDepth rows, `stride` entries each, in shared memory.
struct Lists {
    int32_t *ids;
    float *z;    // the draft's logits of them
    float *lp;   // the target's log-probabilities, or its logits
    float *p;    // and probabilities
    int32_t *hash;
    int stride;
};

constexpr int kListBytes = kDepth * 16, kHashBytes = kHash * 4;  // an entry of a list in every row; the table

// How a call's rows are laid out over the GPU.
struct Plan {
    int32_t cluster;      // CTAs of a row
    int32_t clusters;     // of the grid
    int32_t dynamic;      // a cluster takes its next row when it is free for it (else every clusters-th)
    int32_t eager;        // and at once, rows being short
    int32_t slots;        // of a ring
    int32_t slice_vecs;   // vectors of a slice, but the last's
    int32_t depth_log;    // rows between the scout and the epilogue
    int32_t list_stride;  // entries of a list
    int32_t group_log;    // chunks of a group of top tokens
    int32_t words_at;     // where in shared memory the words of a cluster are
    int32_t smem;
};

}  // namespace token

using namespace token;

namespace {

__device__ __forceinline__ void merge(const TokenParams &P, Part &a, const Part &b) {
    a.n = a.n < 0 || b.n < 0 ? -1 : a.n + b.n;
    if (b.m == -INFINITY) return;
    if (a.m == -INFINITY) {
        a.m = b.m;
        a.s = b.s;
        a.t = b.t;
        return;
    }
    const float m = fmaxf(a.m, b.m);
    float fa, fb;
    const float xa = between(P, a.m, m, fa), xb = between(P, b.m, m, fb);
    a.t = fa * fmaf(xa, a.s, a.t) + fb * fmaf(xb, b.s, b.t);
    a.s = fa * a.s + fb * b.s;
    a.m = m;
}

// The warp's lanes' sums in one, in every lane.
template <class Kd>
__device__ __forceinline__ Part warp_fold(const TokenParams &P, Part a) {
    constexpr uint32_t all = 0xffffffffu;
    Part r;
    r.m = from_order_bits(__reduce_max_sync(all, order_bits(a.m)));
    float f = 0.0f, x = 0.0f;
    if (a.m > -INFINITY) x = between(P, a.m, r.m, f);
    r.s = f * a.s;
    r.t = Kd::Ent && f > 0.0f ? f * fmaf(x, a.s, a.t) : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        r.s += __shfl_xor_sync(all, r.s, off);
        if (Kd::Ent) r.t += __shfl_xor_sync(all, r.t, off);
    }
    r.n = Kd::Rank ? (int)__reduce_add_sync(all, (unsigned)max(a.n, 0)) : 0;
    if (__any_sync(all, a.n < 0)) r.n = -1;
    return r;
}

__device__ __forceinline__ void cluster_arrive(const uint64_t &bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(&bar, rank)) : "memory");
}

// The wait of every role: see wait_on. Most are over at the first look.
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, Shared &S, const TokenParams &P) {
    return wait_on(*static_cast<uint64_t *>(__cvta_shared_to_generic(bar)), parity, S.abort, P.status, P.wait_ns);
}

__device__ __forceinline__ bool wait_at(uint32_t bar, uint32_t parity, Shared &S, const TokenParams &P) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_longer(bar, parity, S, P);
}

__device__ __forceinline__ bool wait_bar(uint64_t &bar, uint32_t parity, Shared &S, const TokenParams &P) {
    return wait_at(smem_u32(&bar), parity, S, P);
}

__device__ __forceinline__ uint4 load_vec(uint32_t at) {
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
    return w;
}

// A CTA's view of the call.
struct Cta {
    int rank, cluster;
    long long first;         // entry
    int slice0, slice_vecs;  // vectors of the row
    int chunks, whole_chunks;  // of the slice; those of nothing but whole vectors, all of them there
    int lane;
    int depth_log;
    uint32_t ring, full, ready, empty;  // in shared memory
    unsigned long long *words;  // what the cluster's warps have sent

    __device__ __forceinline__ int place(int r) const { return r & ((1 << depth_log) - 1); }
    __device__ __forceinline__ uint32_t parity(int r) const { return (uint32_t)r >> depth_log & 1u; }
};

// A place in the ring, and the parity of its barriers' phase.
struct Cursor {
    uint32_t slot = 0, phase = 0;

    __device__ __forceinline__ void step(const Plan &plan) {
        if (++slot == (uint32_t)plan.slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// Sums between the CTAs of a cluster: each number goes with the row's number (of live rows, from 1) in one 8-byte word, so
// that whoever reads it knows that it has come; no barrier, no fence. A warp's words have two places. Row x's replace those
// of row x - 2, which their reader has read: sums of x are sent behind the stores of x - 1, these take sums of x - 1 from
// every CTA, and a CTA sends those behind its own stores of x - 2. (Sums alone: a cluster has one row.)
template <class Kd>
__device__ __forceinline__ unsigned long long *words_of(const Cta &cta, int warp, int live) {
    return cta.words + ((size_t)(live & 1) * cta.cluster * kConsumers + warp) * Kd::kWords;
}

template <class Kd>
__device__ __forceinline__ void send(const Cta &cta, int warp, int live, const Part &p) {
    if (cta.lane >= cta.cluster) return;
    const uint32_t at = cluster_addr(words_of<Kd>(cta, warp, live), cta.lane);
    auto put = [&](int i, uint32_t x) {
        asm volatile("st.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(at + 8 * i),
                     "l"((unsigned long long)(uint32_t)(live + 1) << 32 | x)
                     : "memory");
    };
    put(0, __float_as_uint(p.m));
    put(1, __float_as_uint(p.n < 0 ? NAN : p.s));  // a bad logit
    if (Kd::Ent) put(2, __float_as_uint(p.t));
    if (Kd::Rank) put(2 + Kd::Ent, (uint32_t)p.n);
}

// The cluster's sums of its live-th live row.
template <class Kd>
__device__ bool receive(const TokenParams &P, Shared &S, const Cta &cta, int live, Part &p) {
    p = Part{-INFINITY, 0.0f, 0.0f, 0};
    const uint64_t t0 = global_ns();
    for (int warp = cta.lane; warp - cta.lane < cta.cluster * kConsumers; warp += 32) {
        const uint32_t at = smem_u32(words_of<Kd>(cta, warp, live));
        uint32_t x[Kd::kWords];
        for (;;) {
            bool here = true;
            if (warp < cta.cluster * kConsumers) {
#pragma unroll
                for (int i = 0; i < Kd::kWords; ++i) {
                    unsigned long long w;
                    asm volatile("ld.relaxed.cluster.shared::cta.b64 %0, [%1];" : "=l"(w) : "r"(at + 8 * i) : "memory");
                    x[i] = (uint32_t)w;
                    here = here && (uint32_t)(w >> 32) == (uint32_t)(live + 1);
                }
            }
            if (__all_sync(0xffffffffu, here)) break;
            if (__any_sync(0xffffffffu, *(volatile int32_t *)&S.abort)) return false;
            if (__any_sync(0xffffffffu, global_ns() - t0 > P.wait_ns)) {
                *(volatile int32_t *)&S.abort = 1;
                atomicOr(P.status, SPECVERIFY_STATUS_TIMEOUT);
                return false;
            }
        }
        if (warp < cta.cluster * kConsumers) {
            Part q{__uint_as_float(x[0]), __uint_as_float(x[1]), 0.0f, 0};
            if (Kd::Ent) q.t = __uint_as_float(x[Kd::kWords - 1 - Kd::Rank]);
            if (Kd::Rank) q.n = (int)x[Kd::kWords - 1];
            if (q.s != q.s) {
                q.s = 0.0f;
                q.n = -1;
            }
            merge(P, p, q);
        }
    }
    p = warp_fold<Kd>(P, p);
    return true;
}

// The logits of the row's ragged end, which no copy brings, with -inf behind them.
template <class Kd>
__device__ __forceinline__ uint4 ragged_end(const char *row, int whole, int rest) {
    uint32_t x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        x[q] = Kd::kNegInf;
#pragma unroll
        for (int e = 0; e < 4 / Kd::kSize; ++e) {
            const int at = q * (4 / Kd::kSize) + e;
            if (at >= rest) continue;
            const char *p = row + ((int64_t)whole * Kd::kPer + at) * Kd::kSize;
            if (Kd::DT == SV_DT_FP32) x[q] = *reinterpret_cast<const volatile uint32_t *>(p);
            else x[q] = (x[q] & ~(0xffffu << (16 * e))) | (uint32_t)*reinterpret_cast<const volatile uint16_t *>(p) << (16 * e);
        }
    }
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// What is fetched of an entry ahead of its turn.
struct Asked {
    long long entry;
    int y;
    int64_t row;
    float g, h;
    int id[kMaxList / 32];
    float t[kMaxList / 32];
};

}  // namespace

}  // namespace sv
