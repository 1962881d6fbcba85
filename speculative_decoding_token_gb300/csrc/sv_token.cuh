// sv_token.cuh -- the kernel of the calls on log-probabilities and distillation:
// log-probabilities of given tokens (with entropy, rank and top
// alternatives), the divergence of a draft's rows from its target's top tokens,
// and the gradients of both: one pass over rows of logits.
//
// A row is taken by a cluster of S CTAs, each a slice of it; S = 1 where there
// are rows enough. Slices come in chunks of 16 KiB by bulk copies into a ring of
// shared memory; a gradient's slice comes twice, the second time backwards and
// from L2. The warps of a CTA:
//   consumers (8)  a chunk's vectors, four a thread: the running maximum m, the
//                  sums s of 2^x and t of 2^x x, x = (z - m) log2(e) / T; on the
//                  second reading, with the row's sums known, the gradient;
//   scout          the next row, and what its entry asks for (its token, or its
//                  list with the logits and probabilities of it);
//   producer       the copies;
//   patcher        (lists) takes the listed tokens out of a chunk that has
//                  arrived (-inf), so that the sums are over the rest alone;
//   epilogue       merges the warps' sums (and the cluster's), picks the top
//                  tokens, writes the results, and hands the consumers what a
//                  gradient's second reading needs.
// No warp waits for the end of a row but the consumers of a gradient. Rows are
// taken over from CTAs (clusters) that have not begun, one at a time, when the
// copies of the row before are on their way: CTAs differ by a sixth in speed.
#pragma once

#include "sv_token.h"
#include "sv_rows.cuh"
#include "sv_tree.h"

#include <cuda_bf16.h>

#include <algorithm>

namespace sv {

namespace token {

constexpr int kConsumers = 8;                     // warps
constexpr int kScout = kConsumers, kProducer = kScout + 1, kPatcher = kProducer + 1, kEpilogue = kPatcher + 1;  // (patcher: lists)
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
constexpr int kGroupRows = 20;                    // groups of a thread's vectors in a slice whose maxima are kept
constexpr int kMine = 256, kKept = 512;           // groups that may hold top tokens, a warp's and all
constexpr unsigned kLost = 1u << 24;
constexpr int kKeys = 512;                        // tokens among them
// Keys that a cluster's CTAs send to its first at most: more than a key a lane costs more to put in order than more CTAs save
// (five rows of 32000 fp32 logits, k = 5: 12.8 us in clusters of 4, 13.7 of 8, 16.7 of 16).
constexpr int kGathered = 32;
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
    static constexpr int kEpilogues = Top ? 2 : 1;  // warps that take rows in turn (top tokens take one longer than short sums)
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
    float g, h;    // what the gradient is multiplied by
};

// Sums over part of a row: s of 2^x and t of 2^x x, x = (z - m) c, m a logit
// near the largest (-inf where there is none but -inf); n tokens before the given
// one, -1: a bad logit.
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
    float fix[kDepth];    // the given token's gradient, or what a list's needs
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
    uint16_t kept[kTopDepth][kKept];              // and of all of them, where that was not enough
    unsigned long long keys[kTopDepth][kKeys];
    unsigned long long gathered[kGathered];
    unsigned found[kTopDepth];                    // keys; kLost and more: not all of them
};

// Lists of kDepth rows, `stride` entries each, in shared memory.
struct Lists {
    int32_t *ids;
    float *z;    // the draft's logits of them
    float *lp;   // the target's log-probabilities
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

__device__ __forceinline__ uint32_t order_bits(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 orders as 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float from_order_bits(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ unsigned long long order_key(float v, int i) {
    return ((unsigned long long)order_bits(v) << 32) | (uint32_t)~i;
}

// Logits that the same kernel overwrites later, where a gradient takes their place.
template <int DT>
__device__ __forceinline__ float plain_logit(const char *row, int64_t v) {
    if (DT == SV_DT_FP32) return *reinterpret_cast<const volatile float *>(row + 4 * v);
    return __uint_as_float((uint32_t)*reinterpret_cast<const volatile uint16_t *>(row + 2 * v) << 16);
}

__device__ __forceinline__ uint16_t to_bf16(float x) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
    return h;
}

__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int DT>
__device__ __forceinline__ void store_logit(char *row, int64_t v, float x) {
    if (DT == SV_DT_FP32) reinterpret_cast<float *>(row)[v] = x;
    else reinterpret_cast<uint16_t *>(row)[v] = to_bf16(x);
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Pair i of a vector's logits.
template <int DT>
__device__ __forceinline__ float2 pair_of(const uint4 &w, int i) {
    if (DT == SV_DT_FP32)
        return i == 0 ? make_float2(__uint_as_float(w.x), __uint_as_float(w.y))
                      : make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    const uint32_t x = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    return make_float2(bf16_lo(x), bf16_hi(x));
}

// d / T for a difference d of logits, as a pair of floats
__device__ __forceinline__ void over_T(const TokenParams &P, float hi, float lo, float &rh, float &rl) {
    rh = hi * P.inv_hi;
    rl = 0.0f;
    if (fabsf(rh) < INFINITY) ff_mul(hi, lo, P.inv_hi, P.inv_lo, rh, rl);
}

// ln x of a positive normal x as a pair of floats, to about 2^-25 of one
__device__ __forceinline__ void ff_log(float x, float &h, float &l) {
    uint32_t b = __float_as_uint(x);
    int e = (int)(b >> 23) - 127;
    float f = __uint_as_float((b & 0x007fffffu) | 0x3f800000u);
    if (f > 1.41421356f) {
        f *= 0.5f;
        ++e;
    }
    float eh, el;
    ff_mul((float)e, 0.0f, kLn2Hi, kLn2Lo, eh, el);
    ff_add(eh, el, logf(f), 0.0f, h, l);
}

// ln(2^((z - m) c) / s) = (z - m) / T - ln s, a pair of floats
__device__ __forceinline__ void ff_logprob(const TokenParams &P, float z, float m, float lh, float ll,
                                           float &h, float &l) {
    float d, e, xh, xl;
    two_sum(z, -m, d, e);
    if (!(fabsf(d) < INFINITY)) e = 0.0f;
    over_T(P, d, e, xh, xl);
    if (!(fabsf(xh) < INFINITY)) {
        h = xh;
        l = 0.0f;
        return;
    }
    ff_add(xh, xl, -lh, -ll, h, l);
}

__device__ __forceinline__ float ff_exp(float h, float l) { return h == -INFINITY ? 0.0f : expf(h) * (1.0f + l); }

// 2^(j / 8) as pairs of floats
__device__ const float2 kExp8[8] = {
    {0x1p+0f, 0.0f},
    {0x1.172b84p+0f, -0x1.c15742p-27f},
    {0x1.306fe0p+0f, 0x1.4636e2p-25f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f},
    {0x1.8ace54p+0f, 0x1.15506ep-27f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f},
    {0x1.d5818ep+0f, -0x1.822dbcp-27f},
};

// e^v of v <= 88 as a pair of floats, to about 2^-40 of itself (0 below e^-86): v = n ln 2 / 8 + x, |x| <= ln 2 / 16, the
// series of e^x with its first three terms as pairs, and 2^(n / 8) from the table (Tang's method, see sv_common.cuh).
__device__ __forceinline__ void ff_exp_near(float v, float &h, float &l) {
    h = l = 0.0f;
    if (!(v > -86.0f)) return;
    const float n = rintf(v * 11.5415603f);
    float ph, pl, xh, xl;
    ff_mul(n * 0.125f, 0.0f, kLn2Hi, kLn2Lo, ph, pl);
    ff_add(v, 0.0f, -ph, -pl, xh, xl);
    const float sq = xh * xh, sl = fmaf(xh, xh, -sq) + 2.0f * xh * xl;
    const float tail = sq * xh * fmaf(xh, fmaf(xh, fmaf(xh, 1.0f / 720.0f, 1.0f / 120.0f), 1.0f / 24.0f), 1.0f / 6.0f);
    float eh, el;
    ff_add(xh, xl, 0.5f * sq, fmaf(0.5f, sl, tail), eh, el);
    ff_add(1.0f, 0.0f, eh, el, eh, el);
    const int i = (int)n;
    const float2 t = kExp8[i & 7];
    ff_mul(eh, el, t.x, t.y, h, l);
    const float scale = __uint_as_float((uint32_t)((i >> 3) + 127) << 23);
    h *= scale;
    l *= scale;
}

// e^(h + l) as a pair
__device__ __forceinline__ void ff_exp_pair(float h, float l, float &rh, float &rl) {
    ff_exp_near(h, rh, rl);
    rl = fmaf(rh, l, rl);
}

// ln(x + xl), xl a rounding's worth of x, as a pair of floats good to 2^-40: ff_log's head y, and what x e^-y is more than 1.
__device__ __forceinline__ void ff_log_near(float x, float xl, float &h, float &l) {
    float eh, el;
    ff_log(x, h, l);
    ff_exp_near(-h, eh, el);
    l = fmaf(x, eh, -1.0f) + fmaf(x, el, xl * eh);
}

// a ln(a / b) - a + b, none of it negative, with x = ln(a / b): sums of these have no large terms that cancel. a, b >= 0
__device__ __forceinline__ float divergence_of(float a, float b, float x) {
    if (!(a > 0.0f)) return b;
    if (fabsf(x) > 0.5f) return fmaf(a, x - 1.0f, b);
    // x - 1 + e^-x
    const float c = fmaf(x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, -1.0f / 362880.0f, 1.0f / 40320.0f), -1.0f / 5040.0f),
                                                   1.0f / 720.0f), -1.0f / 120.0f), 1.0f / 24.0f), -1.0f / 6.0f);
    return a * (x * x) * fmaf(x, c, 0.5f);
}

// ln(1 + b (e^r - 1)), good where r is small; 0 < b < 1
__device__ __forceinline__ float ln_mixed(float b, float r) { return r > 40.0f ? r + logf(b) : log1pf(b * expm1f(r)); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    return x;
}

// Logits, and differences of them, are told from -inf down to P.far, -2^25 / c: of no weight either way (with |R| < 2^24), and
// a weight's product with its exponent is 0 and not NaN, also with an entropy's factor between them (below 2^100).

// Of a reference nearer to zero than this, exponents are z c - R with R = m c rounded: one FMA, whose product is exact. |R| <
// 2^24, so that R is off by a half at most, and that is made good in the sum. Others take (z - m) c, with the difference first.
__device__ __forceinline__ bool plain(const TokenParams &P, float m) { return fabsf(m) < P.near; }

// R (rounded: no sum takes the product exactly)
__device__ __forceinline__ float scaled(const TokenParams &P, float m) { return __fmul_rn(m, P.c); }

// What m c is more than the R that is taken of it.
__device__ __forceinline__ float off_by(const TokenParams &P, float m) { return plain(P, m) ? fmaf(m, P.c, -scaled(P, m)) + m * P.c_lo : 0.0f; }

// A thread's reference m is its warp's maximum in the first chunk, and moves when a logit is 8 binades above it
// (TokenParams::lag): the sums are good whatever m is, and moving it for every new maximum costs 30 instructions in nearly
// every chunk (one of 32 lanes has a new maximum). What entropies lose by it is 8 2^-24.

// (z - m) log2(e) / T of a difference
__device__ __forceinline__ float exponent(const TokenParams &P, float d) {
    d = fmaxf(d, P.far);
    return fmaf(d, P.c_lo, d * P.c);
}

// P.far as logits2 takes it
template <int DT>
__device__ __forceinline__ uint32_t far_bits(const TokenParams &P) {
    const uint32_t b = __float_as_uint(P.far);
    return DT == SV_DT_FP32 ? b : b | b >> 16;
}

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
    const float xa = exponent(P, a.m - m), xb = exponent(P, b.m - m);
    const float fa = ex2_approx(xa), fb = ex2_approx(xb);
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
    const float x = exponent(P, a.m - r.m), f = a.m == -INFINITY ? 0.0f : ex2_approx(x);
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

// The j-th largest of the warp's values (j from 1).
__device__ __forceinline__ uint32_t warp_nth(uint32_t x, int j, int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
        for (int i = k >> 1; i > 0; i >>= 1) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, x, i);
            const bool larger = ((lane & k) == 0) == ((lane & i) == 0);
            x = larger ? max(x, o) : min(x, o);
        }
    }
    return __shfl_sync(0xffffffffu, x, j - 1);
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

// ---------------------------------------------------------------------------
// top tokens

// Sorts 32 N keys, the largest first; element 32 q + i is x[q] of lane i (a bitonic network, rolled up: it runs once a row, and
// its instructions would not stay in the cache).
template <int N>
__device__ __forceinline__ void sort_keys(unsigned long long (&x)[N], int lane) {
#pragma unroll 1
    for (int k = 2; k <= 32 * N; k <<= 1) {
#pragma unroll 1
        for (int j = k >> 1; j > 0; j >>= 1) {
            if (j < 32) {
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    const unsigned long long o = __shfl_xor_sync(0xffffffffu, x[q], j);
                    const bool larger = (((32 * q + lane) & k) == 0) == ((lane & j) == 0);
                    x[q] = larger ? max(x[q], o) : min(x[q], o);
                }
                continue;
            }
#pragma unroll
            for (int step = 1; step < N; step <<= 1) {
                if (j != 32 * step) continue;
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    if (q & step) continue;
                    const bool falls = ((32 * q) & k) == 0;
                    const unsigned long long a = max(x[q], x[q ^ step]), b = min(x[q], x[q ^ step]);
                    x[q] = falls ? a : b;
                    x[q ^ step] = falls ? b : a;
                }
            }
        }
    }
}

// The first k of n keys, in order, to the start of them (0 where there are no more); n <= kKeys, k <= 32 N.
template <int N>
__device__ __forceinline__ void sort_front(unsigned long long *keys, int n, int k, int lane) {
    unsigned long long x[N];
#pragma unroll
    for (int q = 0; q < N; ++q) x[q] = 32 * q + lane < n ? keys[32 * q + lane] : 0;
    sort_keys<N>(x, lane);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < N; ++q)
        if (32 * q + lane < k) keys[32 * q + lane] = x[q];
    __syncwarp();
}

__device__ __noinline__ void first_keys(unsigned long long *keys, int n, int k, int lane) {
    if (n <= 32 && k <= 32) sort_front<1>(keys, n, k, lane);
    else if (n <= 64 && k <= 64) sort_front<2>(keys, n, k, lane);
    else if (n <= 128) sort_front<4>(keys, n, k, lane);
    else if (n <= 256) sort_front<8>(keys, n, k, lane);
    else sort_front<kKeys / 32>(keys, n, k, lane);
}

// exclusive sums over the lanes, and the total
__device__ __forceinline__ int lanes_before(int c, int lane, int &total) {
    int incl = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    return incl - c;
}

__device__ __forceinline__ uint32_t gt_mask(uint32_t a, uint32_t b) {
    return __hgt2_mask(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
}

__device__ __forceinline__ uint32_t eq_mask(uint32_t a, uint32_t b) {
    return __heq2_mask(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
}

// What top tokens are chosen from. 8 warps have 8 nth >= k tokens no smaller than the least of their bounds. The bound's class
// are the logits whose upper 16 bits are its own: one value of bf16, 2^-7 of a value of fp32. Tokens above the class are in
// groups above it. Only if they are fewer than k, tokens of the class are needed, of bf16 those of the lowest indexes.
template <int DT>
struct Chooser {
    static constexpr int kPer = 16 / (DT == SV_DT_FP32 ? 4 : 2);
    using Kd = Kind<DT, false, false, true, true, false>;
    const TokenParams &P;
    const char *row;
    const Cta &cta;
    int log;
    uint32_t bound2, high2;
    float low, high;

    __device__ __forceinline__ Chooser(const TokenParams &P_, const Plan &plan, const char *row_, const SharedTop &T, int d, const Cta &cta_)
        : P(P_), row(row_), cta(cta_), log(plan.group_log) {
        const float least = from_order_bits(__reduce_min_sync(0xffffffffu, cta.lane < kConsumers ? T.bound[d][cta.lane] : ~0u));
        const uint32_t bound = __float_as_uint(least) >> 16;
        bound2 = bound | bound << 16;
        low = high = __uint_as_float(bound << 16);
        if (DT == SV_DT_FP32 && fabsf(low) < INFINITY) {
            const float far = __uint_as_float(bound << 16 | 0xffffu);
            if (least < 0.0f) low = far;
            else high = far;
            if ((bound & 0x7fffu) == 0) {  // both zeros' classes are one
                low = __uint_as_float(0x8000ffffu);
                high = __uint_as_float(0x0000ffffu);
            }
        }
        high2 = __float_as_uint(high) >> 16 | (__float_as_uint(high) & 0xffff0000u);
    }

    // Eight groups' maxima: bit 16 (i & 1) + i / 2 for group i above the class, or in it.
    __device__ __forceinline__ uint32_t groups(const uint4 &w, bool equal) const {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
        uint32_t in = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) in |= (equal ? eq_mask(x[q], bound2) : gt_mask(x[q], bound2)) & 0x00010001u << q;
        return in;
    }
    static __device__ __forceinline__ int group_of(uint32_t in) {
        const int bit = __ffs(in) - 1;
        return 2 * (bit & 15) + (bit >> 4);
    }

    // Vector `part` of group g of the slice, -1 past its end.
    __device__ __forceinline__ int vector(int g, int part) const {
        const int v = (((g / kTeam) << log) + (part >> 2)) * Kd::kChunkVecs + (part & 3) * kTeam + g % kTeam;
        return v < cta.slice_vecs ? cta.slice0 + v : -1;
    }

    // Vector v of the row; -inf for what is not there. (No read-only load: the row may have been written while this kernel
    // waited for the one before. Four of them are in flight, past L1: 2000 rows take 138.6 us,
    // 140.6 through it; the ragged end comes after.)
    __device__ __forceinline__ uint4 load(int v) const {
        uint4 w = make_uint4(Kd::kNegInf, Kd::kNegInf, Kd::kNegInf, Kd::kNegInf);
        asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
            : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)
            : "l"(row + (int64_t)v * 16), "r"((uint32_t)(v >= 0 && v < P.V / kPer)));
        return w;
    }
    __device__ __forceinline__ void load_end(uint4 &w, int v) const {
        const int whole = P.V / kPer;
        if (v == whole) w = ragged_end<Kd>(row, whole, P.V - whole * kPer);
    }

    // A vector's tokens above the class, or in it: bit u for token u.
    __device__ __forceinline__ uint32_t tokens(const uint4 &w, int v, bool equal) const {
        uint32_t in = 0;
        if (DT == SV_DT_BF16) {
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) in |= (equal ? eq_mask(x[q], high2) : gt_mask(x[q], high2)) & 0x00020001u << (2 * q);
            in = (in | in >> 16) & 0xffu;
        } else {
            const float x[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
#pragma unroll
            for (int u = 0; u < 4; ++u) in |= (equal ? x[u] >= low && x[u] <= high : x[u] > high) ? 1u << u : 0u;
        }
        if (equal) {  // (what stands in for tokens that are not there is -inf)
            if (v < 0) in = 0;
            else if (P.V - v * kPer < kPer) in &= (1u << (P.V - v * kPer)) - 1u;
        }
        return in;
    }

    // Their keys, from keys[to] on, to keys[end] at most.
    __device__ __forceinline__ void put(unsigned long long *keys, const uint4 &w, int v, uint32_t in, int to, int end) const {
        for (; in; in &= in - 1, ++to) {
            const int u = __ffs(in) - 1;
            const uint32_t x = DT == SV_DT_FP32 ? (u == 0 ? w.x : u == 1 ? w.y : u == 2 ? w.z : w.w)
                                                : (u < 2 ? w.x : u < 4 ? w.y : u < 6 ? w.z : w.w) >> (16 * (u & 1)) << 16;
            if (to < end) keys[to] = order_key(__uint_as_float(x), v * kPer + u);
        }
    }

    // Calls f(vectors, their indexes) over vector index(0) .. index(n - 1), four of a lane at a time, while it says so: read
    // once more from memory (L2).
    template <class Index, class F>
    __device__ __forceinline__ void each(int n, Index &&index, F &&f) const {
        for (int i = 0; i < n; i += 128) {
            uint4 w[4];
            int v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = i + 32 * q + cta.lane;
                v[q] = j < n ? index(j) : -1;
                w[q] = load(v[q]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) load_end(w[q], v[q]);
            if (!f(w, v)) return;
        }
    }
};

// A consumer warp's share of a row's top tokens, once all warps have said their bounds: an eighth of the groups' maxima, and
// the vectors of those above the bound's class read again (of a row of 152064 bf16 logits and k = 64, 115 of 4864 groups and
// 460 vectors; one warp alone took 15 us for it, beside the next row's sums).
template <int DT>
__device__ __noinline__ void gather_top(const TokenParams &P, const Plan &plan, const char *row, SharedTop &T, int d, const Cta cta,
                                        int warp) {
    const Chooser<DT> choose(P, plan, row, T, d, cta);
    const int lane = cta.lane, log = plan.group_log;
    const int pieces = ((cta.chunks + (1 << log) - 1) >> log) * (kTeam / 8);
    uint16_t *mine = T.mine[warp];
    int n = 0;
    for (int i = warp * 32; i < pieces; i += kTeam) {
        uint32_t in = 0;
        if (i + lane < pieces) in = choose.groups(*reinterpret_cast<const uint4 *>(&T.most[d][0][(i + lane) * 8]), false);
        int total, to = lanes_before(__popc(in), lane, total) + n;
        for (; in; in &= in - 1, ++to)
            if (to < kMine) mine[to] = (uint16_t)((i + lane) * 8 + choose.group_of(in));
        n += total;
    }
    __syncwarp();
    if (n > kMine) {
        if (lane == 0) atomicAdd(&T.found[d], kLost);
        return;
    }
    choose.each(n << (2 + log), [&](int j) { return choose.vector(mine[j >> (2 + log)], j & ((4 << log) - 1)); },
                [&](const uint4 (&w)[4], const int (&v)[4]) {
        uint32_t in[4];
        int c = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            in[q] = choose.tokens(w[q], v[q], false);
            c += __popc(in[q]);
        }
        int total, to = lanes_before(c, lane, total);
        if (total == 0) return true;
        unsigned from = 0;
        if (lane == 0) from = atomicAdd(&T.found[d], (unsigned)total);
        to += (int)(__shfl_sync(0xffffffffu, from, 0) & (kLost - 1));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            choose.put(T.keys[d], w[q], v[q], in[q], to, kKeys);
            to += __popc(in[q]);
        }
        return true;
    });
}

// The rest of the choice where the class is needed, or too many tokens are above it: keys to T.keys[d], in any order, and how
// many.
template <int DT>
__device__ __noinline__ int choose_more(const TokenParams &P, const Plan &plan, const char *row, SharedTop &T, int d, const Cta cta,
                                        unsigned found_) {
    const Chooser<DT> choose(P, plan, row, T, d, cta);
    constexpr int kPer = Chooser<DT>::kPer;
    const int lane = cta.lane, k = P.k, log = plan.group_log;
    const int rows = (cta.chunks + (1 << log) - 1) >> log;
    unsigned long long *keys = T.keys[d];
    auto slice = [&](int j) { return cta.slice0 + j; };
    if (found_ < (unsigned)k) {
        // Groups above the class and, chunk after chunk, those in it until there are enough (of fp32: all).
        const int larger = (int)found_;
        int found = larger, groups = 0, equal = 0;
        for (int r = 0; r < rows; ++r) {
            const uint4 w = *reinterpret_cast<const uint4 *>(&T.most[d][r][lane * 8]);
            const bool more = DT == SV_DT_FP32 || equal < k - larger;
            uint32_t in = choose.groups(w, false);
            if (more) {
                const uint32_t same = choose.groups(w, true);
                equal += (int)__reduce_add_sync(0xffffffffu, (unsigned)__popc(same));
                in |= same;
            }
            int total, to = lanes_before(__popc(in), lane, total) + groups;
            for (; in; in &= in - 1, ++to)
                if (to < kKept) T.kept[d][to] = (uint16_t)(r * kTeam + lane * 8 + choose.group_of(in));
            groups += total;
        }
        __syncwarp();
        bool ok = groups <= kKept;
        if (ok)
            choose.each(groups << (2 + log), [&](int j) { return choose.vector(T.kept[d][j >> (2 + log)], j & ((4 << log) - 1)); },
                        [&](const uint4 (&w)[4], const int (&v)[4]) {
                uint32_t in[4];
                int c = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    in[q] = choose.tokens(w[q], v[q], true);
                    c += __popc(in[q]);
                }
                int total, to = lanes_before(c, lane, total) + found;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    choose.put(keys, w[q], v[q], in[q], to, kKeys);
                    to += __popc(in[q]);
                }
                found += total;
                return found <= kKeys;
            });
        __syncwarp();
        if (ok && found <= kKeys) return found;
        if (DT == SV_DT_BF16) {
            // the slice's first tokens that equal the bound, from its start
            found = larger;
            choose.each(cta.slice_vecs, slice, [&](const uint4 (&w)[4], const int (&v)[4]) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t in = choose.tokens(w[q], v[q], true);
                    int total;
                    const int to = lanes_before(__popc(in), lane, total) + found;
                    choose.put(keys, w[q], v[q], in, to, k);
                    found = min(k, found + total);
                }
                return found < k;
            });
            __syncwarp();
            return found;
        }
    }
    // Many tokens within a hair of the bound: the largest key that k of them reach, a bit at a time over the whole slice.
    unsigned long long key = 0;
    int found = 0;
    for (int bit = 63; bit >= -1; --bit) {
        const unsigned long long next = bit < 0 ? key : key | 1ull << bit;
        int c = 0;
        choose.each(cta.slice_vecs, slice, [&](const uint4 (&w)[4], const int (&v)[4]) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float x[kPer];
                vec_floats<DT>(w[q], x);
                uint32_t in = 0;
#pragma unroll
                for (int u = 0; u < kPer; ++u)
                    if (v[q] >= 0 && v[q] * kPer + u < P.V && order_key(x[u], v[q] * kPer + u) >= next) in |= 1u << u;
                if (bit >= 0) {
                    c += __popc(in);
                } else {
                    int total;
                    const int to = lanes_before(__popc(in), lane, total) + found;
                    choose.put(keys, w[q], v[q], in, to, kKeys);
                    found += total;
                }
            }
            return true;
        });
        if (bit >= 0 && (int)__reduce_add_sync(0xffffffffu, (unsigned)c) >= k) key = next;
    }
    __syncwarp();
    return min(found, kKeys);
}

// The k best keys of the CTA's slice, in order, to the start of T.keys[d] (0 where there are none).
template <int DT>
__device__ __forceinline__ void select_top(const TokenParams &P, const Plan &plan, const char *row, SharedTop &T, int d, const Cta &cta) {
    const unsigned found = *(volatile unsigned *)&T.found[d];
    int n = (int)found;
    if (found < (unsigned)P.k || found > (unsigned)kKeys) n = choose_more<DT>(P, plan, row, T, d, cta, found);
    __syncwarp();
    first_keys(T.keys[d], n, P.k, cta.lane);
    if (cta.lane == 0) T.found[d] = 0;  // for the row after the next
}

// ---------------------------------------------------------------------------
// consumers

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The maximum of a vector, NaN if there is one: bf16 as a pair of them, still packed.
template <int DT>
__device__ __forceinline__ uint32_t packed_max(const uint4 &w) {
    if (DT == SV_DT_FP32) return __float_as_uint(vec_max<DT>(w));
    return max_nan_bf16x2(max_nan_bf16x2(w.x, w.y), max_nan_bf16x2(w.z, w.w));
}

template <int DT>
__device__ __forceinline__ uint32_t packed_max(uint32_t a, uint32_t b) {
    if (DT == SV_DT_FP32) return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
    return max_nan_bf16x2(a, b);
}

template <int DT>
__device__ __forceinline__ float from_packed_max(uint32_t x) {
    return DT == SV_DT_FP32 ? __uint_as_float(x) : max_nan(bf16_lo(x), bf16_hi(x));
}

// The largest logit that leaves a reference m where it is (bf16: a pair of it); of one that is no plain number, itself.
template <int DT>
__device__ __forceinline__ uint32_t packed_limit(const TokenParams &P, float m) {
    const float x = plain(P, m) ? m + P.lag : m;
    if (DT == SV_DT_FP32) return __float_as_uint(x);
    // rounded down: a step of bf16 can be hundreds of binades of weight
    const uint32_t b = (__float_as_uint(x) >> 16) + (x < 0.0f && (__float_as_uint(x) & 0xffffu) ? 1u : 0u);
    return b | b << 16;
}

// Whether any of them is larger, or no number.
template <int DT>
__device__ __forceinline__ bool beyond(uint32_t all, uint32_t limit) {
    if (DT == SV_DT_FP32) return !(__uint_as_float(all) <= __uint_as_float(limit));
    return !__hble2(*reinterpret_cast<const __nv_bfloat162 *>(&all), *reinterpret_cast<const __nv_bfloat162 *>(&limit));
}

// Word i of a vector, or pair i of fp32 logits, as two floats; with the entropy, no less than far (bf16: a pair of it).
template <class Kd>
__device__ __forceinline__ f32x2 logits2(const uint4 &w, int i, uint32_t far) {
    if (Kd::DT == SV_DT_FP32) {
        float lo = __uint_as_float(i == 0 ? w.x : w.z), hi = __uint_as_float(i == 0 ? w.y : w.w);
        if (Kd::Ent) {
            lo = fmaxf(lo, __uint_as_float(far));
            hi = fmaxf(hi, __uint_as_float(far));
        }
        return pack2(lo, hi);
    }
    uint32_t x = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    if (Kd::Ent) x = max_bf16x2(x, far);
    return pack2(bf16_lo(x), bf16_hi(x));
}

// The exponents of pair i where the row's maximum is not a plain number.
template <class Kd>
__device__ __forceinline__ f32x2 far_exponents2(const TokenParams &P, const uint4 &w, int i, float m) {
    const float2 z = pair_of<Kd::DT>(w, i);
    return pack2(exponent(P, z.x - m), exponent(P, z.y - m));
}

// Tokens of a vector before the given one (logit zy, token y): those larger, and equal ones of a lower index. first: the
// vector's first token.
template <class Kd>
__device__ __noinline__ int count_before(uint4 w, float zy, int y, int first) {
    int n = 0;
#pragma unroll
    for (int q = 0; q < Kd::kPer / 2; ++q) {
        const float2 z = pair_of<Kd::DT>(w, q);
        n += (z.x > zy || (z.x == zy && first + 2 * q < y)) ? 1 : 0;
        n += (z.y > zy || (z.y == zy && first + 2 * q + 1 < y)) ? 1 : 0;
    }
    return n;
}

// The next lower number of the logits' type; of -inf NaN, which nothing is larger than.
template <int DT>
__device__ __forceinline__ float next_below(float x) {
    constexpr int kShift = DT == SV_DT_FP32 ? 0 : 16;
    const uint32_t b = __float_as_uint(x) >> kShift, sign = 0x80000000u >> kShift;
    const uint32_t r = (b & ~sign) == 0 ? sign | 1u : b & sign ? b + 1 : b - 1;
    return __uint_as_float(r << kShift);
}

// Logits of a vector larger than a bound (bf16: a pair of it). bf16 counts both halves of a word at once: a true half is
// 0xffff, so that a words' sum is 65536 (lo - hi) - lo of the counts of their low and high halves.
template <int DT>
__device__ __forceinline__ uint32_t count_above(const uint4 &w, uint32_t bound) {
    if (DT == SV_DT_FP32) {
        const float t = __uint_as_float(bound);
        return (__uint_as_float(w.x) > t) + (__uint_as_float(w.y) > t) + (__uint_as_float(w.z) > t) + (__uint_as_float(w.w) > t);
    }
    auto above = [&](uint32_t x) {
        return __hgt2_mask(*reinterpret_cast<const __nv_bfloat162 *>(&x), *reinterpret_cast<const __nv_bfloat162 *>(&bound));
    };
    return (above(w.x) + above(w.y)) + (above(w.z) + above(w.w));
}

template <int DT>
__device__ __forceinline__ int counted(uint32_t sum) {
    if (DT == SV_DT_FP32) return (int)sum;
    const uint32_t lo = 0u - sum & 0xffffu;
    return (int)(lo + ((lo - ((sum + lo) >> 16)) & 0xffffu));
}

// The sums of a row's slice, chunk after chunk.
template <class Kd>
__device__ __forceinline__ bool sum_slice(const TokenParams &P, const Plan &plan, Shared &S, SharedTop *top, const Cta &cta, int d,
                                          uint32_t row_parity, int live, Cursor &cur) {
    constexpr int kVecs = Kd::kVecs, kPer = Kd::kPer;
    const int tid = threadIdx.x, lane = cta.lane, warp = tid >> 5;
    float m = -INFINITY, R = -INFINITY;
    uint32_t most = Kd::kNegInf, group = Kd::kNegInf, limit = 0;
    f32x2 s0 = 0ull, s1 = 0ull, t0 = 0ull, t1 = 0ull;
    bool bad = false;
    int before = 0;
    uint32_t above = 0, bound_before = 0, bound_after = 0;
    int y_vec = 0;
    if (Kd::Rank) {
        if (!wait_bar(S.scouted[d], row_parity, S, P)) return false;
        // a token equal to the given one comes before it where its index is lower
        const float zy = S.row[d].zy, below = next_below<Kd::DT>(zy);
        y_vec = S.row[d].y / kPer;
        bound_after = __float_as_uint(zy);
        bound_before = __float_as_uint(below);
        if (Kd::DT == SV_DT_BF16) {
            bound_after |= bound_after >> 16;
            bound_before |= bound_before >> 16;
        }
        if (zy == -INFINITY) bound_before = bound_after;  // and the equal ones one by one, below
    }
    const float c = P.c;
    const f32x2 c2 = pack2(c, c);
    const uint32_t far = far_bits<Kd::DT>(P), mine = cta.ring + tid * 16;
    for (int i = 0; i < cta.chunks; ++i) {
        if (!wait_at(cta.full + 8 * cur.slot, cur.phase, S, P)) return false;
        if (Kd::List && !wait_at(cta.ready + 8 * cur.slot, cur.phase, S, P)) return false;
        const uint32_t at = mine + cur.slot * Kd::kChunkBytes;
        uint4 w[kVecs];
        if (i < cta.whole_chunks) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j) w[j] = load_vec(at + j * kTeam * 16);
        } else {
            const int whole = P.V / kPer, rest = P.V - whole * kPer;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int v = i * Kd::kChunkVecs + tid + j * kTeam;  // of the slice
                w[j] = make_uint4(Kd::kNegInf, Kd::kNegInf, Kd::kNegInf, Kd::kNegInf);
                if (v >= cta.slice_vecs) continue;
                if (!Kd::List && cta.slice0 + v == whole) w[j] = ragged_end<Kd>(S.row[d].z, whole, rest);
                else w[j] = load_vec(at + j * kTeam * 16);
            }
        }
        uint32_t all = packed_max<Kd::DT>(w[0]);
#pragma unroll
        for (int j = 1; j < kVecs; ++j) all = packed_max<Kd::DT>(all, packed_max<Kd::DT>(w[j]));
        if (i == 0 || beyond<Kd::DT>(all, limit)) {
            float cm = from_packed_max<Kd::DT>(all);
            if (!(cm < INFINITY)) {
                bad = true;
                cm = -INFINITY;
                all = Kd::kNegInf;
            }
            if (i == 0) {
                m = from_order_bits(__reduce_max_sync(0xffffffffu, order_bits(cm)));
                R = m == -INFINITY ? -INFINITY : scaled(P, m);
            } else if (cm > m) {
                const float next = scaled(P, cm);
                if (m != -INFINITY) {
                    const float x = plain(P, m) && plain(P, cm) ? R - next : exponent(P, m - cm) - off_by(P, m) + off_by(P, cm);
                    const float f = ex2_approx(x);
                    const f32x2 f2 = pack2(f, f), x2 = pack2(x, x);
                    if (Kd::Ent) {
                        t0 = mul2(f2, fma2(x2, s0, t0));
                        t1 = mul2(f2, fma2(x2, s1, t1));
                    }
                    s0 = mul2(f2, s0);
                    s1 = mul2(f2, s1);
                }
                m = cm;
                R = next;
            }
            limit = packed_limit<Kd::DT>(P, m);
        }
        // The slot is free. Not before the branch above has used all that was loaded: an arrival overtakes loads of shared memory
        // that are queued (behind a gradient's stores), and the slot's next copy with them. (Seen: in gradients of fp32 rows, warps'
        // shares of a chunk from the copy after. A proxy fence instead costs up to 2.5 us of 195.)
        __syncwarp();
        if (lane == 0) mbar_arrive(cta.empty + 8 * cur.slot);
        cur.step(plan);
        if (Kd::Top) {
            // all that the top tokens need of a chunk (lists of the vectors that pass a rising bound took 70 instructions more)
            group = (i & ((1 << plan.group_log) - 1)) == 0 ? all : packed_max<Kd::DT>(group, all);
            most = i == 0 ? all : packed_max<Kd::DT>(most, all);
            top->most[d][i >> plan.group_log][tid] =
                (uint16_t)((Kd::DT == SV_DT_FP32 ? group : max_bf16x2(group, group << 16)) >> 16);
        }
        if (plain(P, m)) {
            const f32x2 nR = pack2(-R, -R);
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
#pragma unroll
                for (int q = 0; q < kPer / 2; ++q) {
                    const f32x2 z2 = logits2<Kd>(w[j], q, far);
                    f32x2 x2 = fma2(z2, c2, nR);
                    if (Kd::List) x2 = fma2(z2, pack2(P.c_lo, P.c_lo), x2);
                    const float2 x = unpack2(x2);
                    const f32x2 e2 = pack2(ex2_approx(x.x), ex2_approx(x.y));
                    if (q & 1) {
                        s1 = add2(s1, e2);
                        if (Kd::Ent) t1 = fma2(e2, x2, t1);
                    } else {
                        s0 = add2(s0, e2);
                        if (Kd::Ent) t0 = fma2(e2, x2, t0);
                    }
                }
        } else if (m != -INFINITY) {
#pragma unroll 1
            for (int j = 0; j < kVecs; ++j) {
                const uint4 v = j == 0 ? w[0] : j == 1 ? w[1] : j == 2 ? w[2] : w[3];
#pragma unroll
                for (int q = 0; q < kPer / 2; ++q) {
                    const f32x2 x2 = far_exponents2<Kd>(P, v, q, m);
                    const float2 x = unpack2(x2);
                    const f32x2 e2 = pack2(ex2_approx(x.x), ex2_approx(x.y));
                    s0 = add2(s0, e2);
                    if (Kd::Ent) t0 = fma2(e2, x2, t0);
                }
            }
        }
        if (Kd::Rank) {
            const int v0 = cta.slice0 + i * Kd::kChunkVecs + tid;
            const bool inf = bound_before == bound_after;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int v = v0 + j * kTeam;
                if (v == y_vec || (inf && v < y_vec)) {
                    if (v < cta.slice0 + cta.slice_vecs) before += count_before<Kd>(w[j], S.row[d].zy, S.row[d].y, v * kPer);
                } else {
                    above += count_above<Kd::DT>(w[j], v < y_vec ? bound_before : bound_after);
                }
            }
            if ((i & 1023) == 1023) {  // what is packed into half a word does not overflow
                before += counted<Kd::DT>(above);
                above = 0;
            }
        }
    }
    if (Kd::Top) {
        // Each warp bounds the k-th largest logit by the nth largest of its lanes' maxima: 8 warps have 8 nth >= k tokens that
        // large.
        const uint32_t nth = warp_nth(order_bits(from_packed_max<Kd::DT>(most)), (P.k + kConsumers - 1) / kConsumers, lane);
        if (lane == 0) top->bound[d][warp] = nth;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&S.bounded[d]));
    }
    const float2 a = unpack2(s0), b = unpack2(s1), e = unpack2(t0), f = unpack2(t1);
    if (Kd::Rank) before += counted<Kd::DT>(above);
    Part p{m, (a.x + a.y) + (b.x + b.y), (e.x + e.y) + (f.x + f.y), bad ? -1 : before};
    if (plain(P, m)) {  // what R was off by
        const float r = off_by(P, m), g = ex2_approx(-r);
        p.t = g * fmaf(-r, p.s, p.t);
        p.s *= g;
    }
    p = warp_fold<Kd>(P, p);
    if constexpr (Kd::Top) {
        if (!wait_bar(S.bounded[d], row_parity, S, P)) return false;
        gather_top<Kd::DT>(P, plan, S.row[d].z, *top, d, cta, warp);
    }
    // (a list's or a token's logits are read before any CTA can overwrite the row)
    if (Kd::Grad && cta.cluster > 1 && !wait_bar(S.scouted[d], row_parity, S, P)) return false;
    if (cta.cluster > 1) send<Kd>(cta, cta.rank * kConsumers + warp, live, p);
    else if (lane == 0) S.part[d][warp] = p;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&S.summed[d]));
    return true;
}

// The gradient of a row's slice, 2^x (a + b x) for x = (z - m) c, the last chunk first.
template <class Kd>
__device__ __forceinline__ bool store_slice(const TokenParams &P, const Plan &plan, Shared &S, const Cta &cta, int d,
                                            uint32_t row_parity, Cursor &cur) {
    constexpr int kPer = Kd::kPer, kVecs = Kd::kVecs;
    const int tid = threadIdx.x, lane = cta.lane;
    const int state = S.row[d].state;
    uint4 *out = reinterpret_cast<uint4 *>(P.grad + S.row[d].entry * P.grad_stride_bytes) + cta.slice0 + tid;
    float m = 0.0f, fa = state == kBad ? NAN : 0.0f, fb = 0.0f;
    if (state == kLive) {
        if (!wait_bar(S.known[d], row_parity, S, P)) return false;
        const float4 cf = S.coef[d];
        m = cf.x;
        fa = cf.y;
        fb = cf.z;
    }
    const float c = P.c, R = scaled(P, m);
    const bool near = plain(P, m);
    constexpr bool kFine = Kd::List && Kd::DT == SV_DT_FP32;  // bf16 gradients have no use for c_lo
    if (near) {
        const float r = kFine ? off_by(P, m) : fmaf(m, c, -R), g = ex2_approx(-r);
        fa = g * fmaf(-r, fb, fa);
        fb *= g;
    }
    const f32x2 nR = pack2(-R, -R), c2 = pack2(c, c), a2 = pack2(fa, fa), b2 = pack2(fb, fb);
    auto exponents = [&](f32x2 z2) {
        const f32x2 x2 = fma2(z2, c2, nR);
        return kFine ? fma2(z2, pack2(P.c_lo, P.c_lo), x2) : x2;
    };
    auto weigh = [&](f32x2 x2) {
        const float2 x = unpack2(x2);
        return mul2(pack2(ex2_approx(x.x), ex2_approx(x.y)), Kd::Ent ? fma2(b2, x2, a2) : a2);
    };
    auto packed = [&](const f32x2 (&g)[kPer / 2]) {
        const float2 x = unpack2(g[0]), y = unpack2(g[1]);
        if (Kd::DT == SV_DT_FP32)
            return make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
        const float2 z = unpack2(g[2 % (kPer / 2)]), u = unpack2(g[3 % (kPer / 2)]);
        return make_uint4(to_bf16x2(x.x, x.y), to_bf16x2(y.x, y.y), to_bf16x2(z.x, z.y), to_bf16x2(u.x, u.y));
    };
    const uint32_t far = far_bits<Kd::DT>(P), mine = cta.ring + tid * 16;
    for (int i = cta.chunks - 1; i >= 0; --i) {
        uint32_t at = mine;
        if (state == kLive) {
            if (!wait_at(cta.full + 8 * cur.slot, cur.phase, S, P)) return false;
            if (Kd::List && !wait_at(cta.ready + 8 * cur.slot, cur.phase, S, P)) return false;
            at += cur.slot * Kd::kChunkBytes;
        }
        uint4 *to = out + i * Kd::kChunkVecs;
        if (state == kLive && near && i < cta.whole_chunks) {
            uint4 w[kVecs];
#pragma unroll
            for (int j = 0; j < kVecs; ++j) w[j] = load_vec(at + j * kTeam * 16);
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                f32x2 g[kPer / 2];
#pragma unroll
                for (int q = 0; q < kPer / 2; ++q) g[q] = weigh(exponents(logits2<Kd>(w[j], q, far)));
                to[j * kTeam] = packed(g);
            }
            __syncwarp();  // (after the stores, which have used the loads: see sum_slice)
            if (lane == 0) mbar_arrive(cta.empty + 8 * cur.slot);
        } else {
            const int whole = P.V / kPer, rest = P.V - whole * kPer;
#pragma unroll 1
            for (int j = 0; j < kVecs; ++j) {
                const int v = i * Kd::kChunkVecs + tid + j * kTeam;  // of the slice
                if (v >= cta.slice_vecs) break;
                const bool end = cta.slice0 + v >= whole;
                f32x2 g[kPer / 2];
                if (state == kLive) {
                    const uint4 w = end ? ragged_end<Kd>(S.row[d].z, whole, rest) : load_vec(at + j * kTeam * 16);
#pragma unroll
                    for (int q = 0; q < kPer / 2; ++q)
                        g[q] = weigh(near ? exponents(logits2<Kd>(w, q, far)) : far_exponents2<Kd>(P, w, q, m));
                } else {
#pragma unroll
                    for (int q = 0; q < kPer / 2; ++q) g[q] = a2;
                }
                if (!end) {
                    to[j * kTeam] = packed(g);
                } else {
#pragma unroll
                    for (int q = 0; q < kPer; ++q) {
                        const float2 x = unpack2(g[q / 2]);
                        if (q < rest) store_logit<Kd::DT>(reinterpret_cast<char *>(to + j * kTeam), q, q & 1 ? x.y : x.x);
                    }
                }
            }
            if (state == kLive) {
                __syncwarp();
                if (lane == 0) mbar_arrive(cta.empty + 8 * cur.slot);
            }
        }
        if (state == kLive) cur.step(plan);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&S.stored[d]));
    return true;
}

template <class Kd>
__device__ __forceinline__ void consume(const TokenParams &P, const Plan &plan, Shared &S, SharedTop *top, const Cta &cta) {
    Cursor cur;
    int live = 0;
    for (int r = 0;; ++r) {
        const int d = cta.place(r);
        if (!wait_bar(S.row_full[d], cta.parity(r), S, P)) return;
        const int state = S.row[d].state;
        if (state == kEnd) return;
        if (state == kLive) {
            if (!sum_slice<Kd>(P, plan, S, top, cta, d, cta.parity(r), live++, cur)) return;
        } else if (cta.lane == 0) {
            if (Kd::Top) mbar_arrive(smem_u32(&S.bounded[d]));
            mbar_arrive(smem_u32(&S.summed[d]));
        }
        if (Kd::Grad && !store_slice<Kd>(P, plan, S, cta, d, cta.parity(r), cur)) return;
        __syncwarp();
        if (cta.lane == 0) mbar_arrive(smem_u32(&S.row_free[d]));
    }
}

// ---------------------------------------------------------------------------
// scout

// The rows of a cluster, one after another. Dynamic: the grid has a cluster for every row, and one that runs takes over, one
// at a time, the rows of those that have not begun (cluster launch control). The first CTA asks, the answer goes to all of
// them, and the next is asked for when they all have read it.
struct Entries {
    long long e;
    int answers, awaited;

    // e < 0 after the last one; false: gave up
    __device__ __forceinline__ bool next(const TokenParams &P, const Plan &plan, Shared &S, const Cta &cta) {
        if (!plan.dynamic) {
            e += plan.clusters;
            if (e >= P.entries) e = -1;
            return true;
        }
        if (cta.rank == 0) {
            if (cta.cluster > 1 && answers > 0 && !wait_bar(S.acked, (uint32_t)(answers - 1) & 1u, S, P)) return false;
            if (cta.lane == 0) {
                S.asked = answers + 1;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                if (cta.cluster == 1)
                    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                                     smem_u32(&S.grant)),
                                 "r"(smem_u32(&S.granted))
                                 : "memory");
                else
                    asm volatile(
                        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 "
                        "[%0], [%1];" ::"r"(smem_u32(&S.grant)),
                        "r"(smem_u32(&S.granted))
                        : "memory");
            }
        }
        if (cta.lane == 0) mbar_arrive_expect_tx(smem_u32(&S.granted), 16);
        ++awaited;
        if (!wait_bar(S.granted, (uint32_t)answers & 1u, S, P)) return false;
        ++answers;
        uint32_t more, x;
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
            "ld.shared.b128 r, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t"
            "mov.u32 %1, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
            : "=r"(more), "=r"(x)
            : "r"(smem_u32(&S.grant))
            : "memory");
        if (cta.cluster > 1) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the next answer comes after this one was read
            __syncwarp();
            if (cta.lane == 0) cluster_arrive(S.acked, 0);
        }
        __syncwarp();
        e = more ? (long long)(x / (uint32_t)cta.cluster) : -1;
        return true;
    }
};

// What is fetched of an entry ahead of its turn.
struct Asked {
    long long entry;
    int y;
    int64_t row;
    float g, h;
    int id[kMaxList / 32];
    float t[kMaxList / 32];
};

template <bool LIST>
__device__ __forceinline__ void fetch(const TokenParams &P, long long e, int lane, Asked &a) {
    if (LIST) {
#pragma unroll
        for (int i = 0; i < kMaxList / 32; ++i) {
            const int j = lane + 32 * i;
            if (j >= P.K) continue;
            a.id[i] = P.ids[e * P.K + j];
            a.t[i] = P.target_bf16 ? plain_logit<SV_DT_BF16>(P.target, e * P.K + j) : plain_logit<SV_DT_FP32>(P.target, e * P.K + j);
        }
        a.g = P.weight ? P.weight[e] : 1.0f;
    } else {
        a.entry = e;
        a.row = e;
        if (P.row_off) {
            // first tokens first: the ends of short sequences, which ask for nothing, come together at the end (in the
            // sequences' order a CTA met several of them, 1.7 us each, before its first row)
            const int b = (int)(e % P.B), m = (int)(e / P.B);
            a.entry = (long long)b * P.M + m;
            const int at = P.path ? P.path[a.entry] : m;
            a.row = at < 0 ? -1 : P.row_off[b] + at;
        }
        a.y = P.tokens[a.entry];
        if (P.grad) {
            a.g = P.g_logprob[e];
            a.h = P.g_entropy ? P.g_entropy[e] : 0.0f;
        }
    }
}

// What a row is: one lane's work.
__device__ __forceinline__ void scout_row(const TokenParams &P, Row &row, const Asked &a) {
    int bits = 0;
    if (a.y != -1) {
        if (a.y < 0 || a.y >= P.V) bits = SPECVERIFY_STATUS_BAD_TOKEN;
        else if (a.row < 0 || a.row >= P.rows) bits = SPECVERIFY_STATUS_BAD_ROW;
    }
    row.z = P.logits + a.row * P.stride_bytes;
    row.entry = a.entry;
    row.y = a.y;
    row.state = a.y == -1 ? kSkip : bits ? kBad : kLive;
    row.g = a.g;
    row.h = a.h;
    if (bits) atomicOr(P.status, bits);
}

// The same of a list, the warp's work: its ids, where they are tokens.
__device__ __forceinline__ void scout_ids(const TokenParams &P, Row &row, const Lists &L, int d, long long e, int lane, const Asked &a) {
    constexpr uint32_t all = 0xffffffffu;
    bool bad = false, any = false;
#pragma unroll
    for (int i = 0; i < kMaxList / 32; ++i) {
        const int j = lane + 32 * i;
        if (j >= P.K) continue;
        const int id = a.id[i];
        const bool token = id >= 0 && id < P.V;
        bad = bad || (!token && id != -1);
        any = any || token;
        L.ids[d * L.stride + j] = token ? id : -1;
    }
    bad = __any_sync(all, bad);
    any = __any_sync(all, any);
    if (lane == 0) {
        row.z = P.logits + e * P.stride_bytes;
        row.entry = e;
        row.state = bad ? kBad : any ? kLive : kSkip;
        row.g = a.g;
        if (bad) atomicOr(P.status, SPECVERIFY_STATUS_BAD_TOKEN);
    }
}

// The rest of a list: the draft's logits of it, the target's log-probabilities, what can be summed of both.
template <int DT>
__device__ __forceinline__ void scout_list(const TokenParams &P, Row &row, const Lists &L, int d, long long e, int lane, const Asked &a) {
    constexpr uint32_t all = 0xffffffffu;
    const char *z = P.logits + e * P.stride_bytes;
    const int32_t *ids = L.ids + d * L.stride;
    float *lz = L.z + d * L.stride, *llp = L.lp + d * L.stride, *lpr = L.p + d * L.stride;
    int bits = 0;
    float top = -INFINITY, zmax = -INFINITY;
    float zk[kMaxList / 32];
#pragma unroll
    for (int i = 0; i < kMaxList / 32; ++i) {
        const int j = lane + 32 * i;
        zk[i] = j < P.K && ids[j] >= 0 ? plain_logit<DT>(z, ids[j]) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kMaxList / 32; ++i) {
        const int j = lane + 32 * i;
        if (j >= P.K) continue;
        const int id = ids[j];
        float t = -INFINITY;
        if (id >= 0) {
            t = a.t[i];
            if (!(zk[i] < INFINITY) || !(t < INFINITY)) bits |= SPECVERIFY_STATUS_BAD_LOGIT;
            // twice the same id: one of its entries finds the other in the table
            uint32_t at = (uint32_t)id * 2654435761u >> 22;
            for (int tries = 0; tries < kHash; ++tries, at = (at + 1) % kHash) {
                const int was = atomicCAS(&L.hash[at], -1, id);
                if (was == id) bits |= SPECVERIFY_STATUS_BAD_TOKEN;
                if (was == -1 || was == id) break;
            }
        }
        lz[j] = zk[i];
        llp[j] = t;
        top = fmaxf(top, t);
        zmax = fmaxf(zmax, zk[i]);
    }
    __syncwarp();
    for (int j = lane; j < kHash / 4; j += 32) reinterpret_cast<int4 *>(L.hash)[j] = make_int4(-1, -1, -1, -1);
    bits = __reduce_or_sync(all, bits);
    float p_rest = 0.0f, p_rest_l = 0.0f, rest_h = -INFINITY, rest_l = 0.0f, over = 0.0f, p0 = 0.0f, p0_l = 0.0f, lp0 = 0.0f, zsum = 0.0f, zsum_l = 0.0f, cross = 0.0f;
    const bool rkl = P.divergence == SPECVERIFY_RKL;
    zmax = warp_max(zmax);
    if (!bits) {
        if (P.form == SPECVERIFY_TARGET_LOGITS) {
            top = warp_max(top);
            float sum = 0.0f, lh = 0.0f, ll = 0.0f;
            for (int j = lane; j < P.K; j += 32) {
                float h, l;
                ff_logprob(P, llp[j], top, 0.0f, 0.0f, h, l);
                sum += llp[j] == -INFINITY ? 0.0f : ff_exp(h, l);
            }
            sum = warp_sum(sum);
            if (top == -INFINITY) bits = SPECVERIFY_STATUS_BAD_LOGIT;  // a target of nothing
            else ff_log(sum, lh, ll);
            for (int j = lane; j < P.K; j += 32) {
                float h, l;
                ff_logprob(P, llp[j], top, lh, ll, h, l);
                if (llp[j] == -INFINITY) h = -INFINITY;
                llp[j] = h;
                lpr[j] = ff_exp(h, 0.0f);
            }
        } else {
            // One less a sum close to it: in pairs of floats, or little would be left of it.
            float sh = 0.0f, sl = 0.0f;
            for (int j = lane; j < P.K; j += 32) {
                float h, l;
                ff_exp_near(llp[j], h, l);
                lpr[j] = h;
                ff_add(sh, sl, h, l, sh, sl);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                ff_add(sh, sl, __shfl_xor_sync(all, sh, off), __shfl_xor_sync(all, sl, off), sh, sl);
            ff_add(1.0f, 0.0f, -sh, -sl, sh, sl);
            p_rest = fmaxf(sh + sl, 0.0f);
            const float least = rkl ? fmaxf(p_rest, 0x1p-20f) : p_rest;
            const bool kept = least == sh + sl;
            p_rest_l = kept ? (sh - least) + sl : 0.0f;
            if (least > 0.0f) ff_log_near(least, p_rest_l, rest_h, rest_l);
            over = kept ? 0.0f : (least - sh) - sl;
        }
        if (zmax > -INFINITY) {
            if (rkl) {
                float mine = -INFINITY;  // ln p of a token with the largest logit
                for (int j = lane; j < P.K; j += 32)
                    if (lz[j] == zmax) mine = fmaxf(mine, llp[j]);
                lp0 = warp_max(mine);
                if (!(lp0 > -80.0f)) lp0 = 0.0f;  // (any number would do)
                ff_exp_near(lp0, p0, p0_l);
            }
            for (int j = lane; j < P.K; j += 32) {
                float d, e, xh, xl, wh, wl;
                two_sum(lz[j], -zmax, d, e);
                if (!(d > P.far)) continue;
                over_T(P, d, e, xh, xl);
                ff_exp_pair(xh, xl, wh, wl);
                ff_add(zsum, zsum_l, wh, wl, zsum, zsum_l);
                if (wh > 0.0f && rkl) {
                    two_sum(llp[j], -lp0, d, e);
                    if (!(fabsf(d) < INFINITY)) e = 0.0f;
                    cross += wh * ((xh - d) + (xl - e));
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            ff_add(zsum, zsum_l, __shfl_xor_sync(all, zsum, off), __shfl_xor_sync(all, zsum_l, off), zsum, zsum_l);
        if (rkl) cross = warp_sum(cross);
    }
    if (lane == 0) {
        row.bad = bits;
        row.p_rest = p_rest;
        row.p_rest_l = p_rest_l;
        row.rest_h = rest_h;
        row.rest_l = rest_l;
        row.over = over;
        row.zmax = zmax;
        row.p0 = p0;
        row.p0_l = p0_l;
        row.lp0 = lp0;
        row.zsum = zsum;
        row.zsum_l = zsum_l;
        row.cross = cross;
        if (bits) atomicOr(P.status, bits);
    }
}

template <class Kd>
__device__ __forceinline__ void scout(const TokenParams &P, const Plan &plan, Shared &S, const Lists &list, const Cta &cta,
                                      Entries &at) {
    Asked a;
    int ends = 0;
    for (int r = 0;; ++r) {
        const int d = cta.place(r);
        if (at.e >= 0) fetch<Kd::List>(P, at.e, cta.lane, a);
        if (!wait_bar(S.row_free[d], cta.parity(r) ^ 1u, S, P)) return;
        if (at.e < 0) {
            if (cta.lane == 0) S.row[d].state = kEnd;
        } else if (Kd::List) {
            scout_ids(P, S.row[d], list, d, at.e, cta.lane, a);
        } else if (cta.lane == 0) {
            scout_row(P, S.row[d], a);
        }
        __syncwarp();
        if (cta.lane == 0) mbar_arrive(smem_u32(&S.row_full[d]));
        if (at.e < 0) {
            if (++ends == Kd::kEpilogues) return;
            continue;
        }
        // The copies can begin; what else there is to know of the entry
        if (S.row[d].state == kLive) {
            if (Kd::List) scout_list<Kd::DT>(P, S.row[d], list, d, at.e, cta.lane, a);
            else if (cta.lane == 0) S.row[d].zy = plain_logit<Kd::DT>(S.row[d].z, a.y);
        }
        __syncwarp();
        if (cta.lane == 0) mbar_arrive(smem_u32(&S.scouted[d]));
        // The next row is asked for when (nearly) all of this one's copies have been issued: not sooner than it is needed.
        if (!plan.eager && !wait_bar(S.sent[d], cta.parity(r), S, P)) return;
        if (!at.next(P, plan, S, cta)) return;
    }
}

// ---------------------------------------------------------------------------
// producer and patcher

template <class Kd>
__device__ __forceinline__ void produce(const TokenParams &P, const Plan &plan, Shared &S, const Cta &cta) {
    const int64_t row_bytes = (int64_t)P.V * Kd::kSize & ~15ll;
    Cursor cur;
    long long issued = 0;
    bool ok = true;
    for (int r = 0;; ++r) {
        const int d = cta.place(r);
        ok = wait_bar(S.row_full[d], cta.parity(r), S, P);
        if (!ok || S.row[d].state == kEnd) break;
        const char *z = S.row[d].z;
        const int n = S.row[d].state != kLive ? 0 : Kd::Grad ? 2 * cta.chunks : cta.chunks;
        const int ask = n == 0 ? -1 : max(0, n - 1 - kLead);
        for (int j = 0; j < n; ++j) {
            ok = wait_at(cta.empty + 8 * cur.slot, cur.phase ^ 1u, S, P);
            if (!ok) break;
            if (cta.lane == 0) {
                const int i = j < cta.chunks ? j : 2 * cta.chunks - 1 - j;  // backwards the second time
                const int64_t off = ((int64_t)cta.slice0 + (int64_t)i * Kd::kChunkVecs) * 16;
                const int most = min(Kd::kChunkVecs, cta.slice_vecs - i * Kd::kChunkVecs) * 16;
                const int bytes = (int)min((int64_t)most, row_bytes - off);
                const uint32_t bar = cta.full + 8 * cur.slot;
                if (bytes > 0) {
                    mbar_arrive_expect_tx(bar, (uint32_t)bytes);
                    bulk_load(cta.ring + cur.slot * Kd::kChunkBytes, z + off, (uint32_t)bytes, bar);
                } else {
                    mbar_arrive(bar);
                }
            }
            ++issued;
            cur.step(plan);
            if (j == ask && cta.lane == 0) mbar_arrive(smem_u32(&S.sent[d]));
        }
        if (!ok) break;
        __syncwarp();
        if (cta.lane == 0) {
            if (ask < 0) mbar_arrive(smem_u32(&S.sent[d]));
            mbar_arrive(smem_u32(&S.row_free[d]));
        }
    }
    // no copy outlives its CTA, also where those who needed it gave up
    for (long long u = max(0ll, issued - plan.slots); u < issued; ++u)
        mbar_wait_bounded(cta.full + 8 * (uint32_t)(u % plan.slots), u / plan.slots & 1);
}

template <class Kd>
__device__ __forceinline__ void patch(const TokenParams &P, const Plan &plan, Shared &S, const Lists &L, uint8_t *ring,
                                      const Cta &cta) {
    const int whole = P.V / Kd::kPer, rest = P.V - whole * Kd::kPer;
    Cursor cur;
    for (int r = 0;; ++r) {
        const int d = cta.place(r);
        if (!wait_bar(S.row_full[d], cta.parity(r), S, P)) return;
        if (S.row[d].state == kEnd) return;
        const int n = S.row[d].state != kLive ? 0 : Kd::Grad ? 2 * cta.chunks : cta.chunks;
        for (int i = 0; i < n; ++i) {
            if (!wait_at(cta.full + 8 * cur.slot, cur.phase, S, P)) return;
            if (i < cta.chunks) {  // the gradient's second reading takes the chunk as it is
                uint8_t *chunk = ring + (size_t)cur.slot * Kd::kChunkBytes;
                const int v0 = cta.slice0 + i * Kd::kChunkVecs;
                const int vecs = min(Kd::kChunkVecs, cta.slice_vecs - i * Kd::kChunkVecs);
                if (rest && v0 <= whole && whole < v0 + vecs) {  // the ragged end of the row, which no copy brings
                    if (cta.lane < Kd::kPer) {
                        const float x =
                            cta.lane < rest ? plain_logit<Kd::DT>(S.row[d].z, (int64_t)whole * Kd::kPer + cta.lane) : -INFINITY;
                        store_logit<Kd::DT>(reinterpret_cast<char *>(chunk + (whole - v0) * 16), cta.lane, x);
                    }
                    __syncwarp();
                }
                for (int j = cta.lane; j < P.K; j += 32) {
                    const int at = L.ids[d * L.stride + j] - v0 * Kd::kPer;
                    if (at >= 0 && at < vecs * Kd::kPer) store_logit<Kd::DT>(reinterpret_cast<char *>(chunk), at, -INFINITY);
                }
                // the next copy into this slot comes after these stores
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            if (cta.lane == 0) mbar_arrive(cta.ready + 8 * cur.slot);
            cur.step(plan);
        }
        __syncwarp();
        if (cta.lane == 0) mbar_arrive(smem_u32(&S.row_free[d]));
    }
}

// ---------------------------------------------------------------------------
// epilogue

template <int DT>
__device__ __forceinline__ void write_top(const TokenParams &P, long long e, int i, unsigned long long key, float m, float lh, float ll) {
    float lp = -INFINITY, lo = 0.0f;
    int idx = -1;
    if (key) {
        idx = (int)~(uint32_t)key;
        ff_logprob(P, from_order_bits((uint32_t)(key >> 32)), m, lh, ll, lp, lo);
    }
    P.top_logprob[e * P.k + i] = lp;
    P.top_idx[e * P.k + i] = idx;
}

template <class Kd>
__device__ __forceinline__ bool finish_token(const TokenParams &P, const Plan &plan, Shared &S, SharedTop *T, const Cta &cta, int d, const Part &p) {
    const Row &row = S.row[d];
    const long long e = row.entry;
    const int lane = cta.lane, k = Kd::Top ? P.k : 0;
    const bool alone = cta.cluster == 1;
    const bool bad = row.state == kBad || (row.state == kLive && (p.n < 0 || p.m == -INFINITY));
    const bool good = row.state == kLive && !bad;
    if (row.state == kLive && bad && lane == 0 && cta.rank == 0) atomicOr(P.status, SPECVERIFY_STATUS_BAD_LOGIT);
    float lh = 0.0f, ll = 0.0f, lp = 0.0f, lo = 0.0f, H = 0.0f;
    const float inv_s = 1.0f / p.s;
    // p_v (-(g + h (ln p_v + H)) / T) with p_v = 2^x / s and ln p_v = x ln 2 - ln s
    if (Kd::Grad && !Kd::Ent && lane == 0) {
        S.coef[d] = good ? make_float4(p.m, -row.g * P.inv_hi * inv_s, 0.0f, 0.0f) : make_float4(0.0f, NAN, 0.0f, 0.0f);
        mbar_arrive(smem_u32(&S.known[d]));
    }
    if (good) {
        ff_log(p.s, lh, ll);
        if (Kd::Ent) {
            const float mean = p.t / p.s;
            H = lh - fmaf(mean, kLn2Hi, fmaf(mean, kLn2Lo, -ll));
        }
    }
    if (Kd::Grad && Kd::Ent && lane == 0) {
        const float a = -(row.g + row.h * (H - lh)) * P.inv_hi * inv_s, b = -row.h * P.inv_hi * kLn2Hi * inv_s;
        S.coef[d] = good ? make_float4(p.m, a, b, 0.0f) : make_float4(0.0f, NAN, NAN, 0.0f);
        mbar_arrive(smem_u32(&S.known[d]));
    }
    if (good) ff_logprob(P, row.zy, p.m, lh, ll, lp, lo);
    else if (bad) lp = H = NAN;
    if (lane == 0 && cta.rank == 0) {
        if (P.logprob) P.logprob[e] = lp;
        if (P.entropy) P.entropy[e] = H;
        if (!Kd::Grad && P.lse) {
            float xh = 0.0f, xl = 0.0f;
            if (good) {
                over_T(P, p.m, 0.0f, xh, xl);
                if (fabsf(xh) < INFINITY) ff_add(xh, xl, lh, ll, xh, xl);
            }
            P.lse[e] = bad ? NAN : xh;
        }
        if (Kd::Rank) P.rank[e] = bad ? -1 : p.n;
    }
    if constexpr (Kd::Top) {
        if (row.state == kLive) {
            select_top<Kd::DT>(P, plan, row.z, *T, d, cta);
            if (!alone) {
                for (int i = lane; i < k; i += 32)
                    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(cluster_addr(&T->gathered[cta.rank * k + i], 0)),
                                 "l"(T->keys[d][i])
                                 : "memory");
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                __syncwarp();
                if (lane == 0) cluster_arrive(S.gathered, 0);
                if (cta.rank != 0) return true;
                if (!wait_bar(S.gathered, 0, S, P)) return false;  // a cluster of such rows has one
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                first_keys(T->gathered, cta.cluster * k, k, lane);
            }
        }
        if (cta.rank != 0) return true;
        const unsigned long long *best = alone ? T->keys[d] : T->gathered;
        for (int i = lane; i < k; i += 32) {
            if (good) {
                write_top<Kd::DT>(P, e, i, best[i], p.m, lh, ll);
            } else {
                P.top_logprob[e * k + i] = bad ? NAN : -INFINITY;
                P.top_idx[e * k + i] = -1;
            }
        }
    }
    if (Kd::Grad && lane == 0) {
        const float py = ff_exp(lp, lo);
        const float s = Kd::Ent && py > 0.0f ? row.h * py * (lp + H) : 0.0f;
        S.fix[d] = (row.g * (1.0f - py) - s) * P.inv_hi;
        S.good[d] = good;
    }
    return true;
}

// Puts the given token's gradient in its place, once the consumers have stored the others'.
template <class Kd>
__device__ __forceinline__ void fix_token(const TokenParams &P, const Shared &S, const Cta &cta, int d) {
    const int y = S.row[d].y, v = y / Kd::kPer;
    if (cta.lane == 0 && S.good[d] && v >= cta.slice0 && v < cta.slice0 + cta.slice_vecs)
        store_logit<Kd::DT>(P.grad + S.row[d].entry * P.grad_stride_bytes, y, S.fix[d]);
}

// The same for a list's tokens.
template <class Kd>
__device__ __forceinline__ void fix_list(const TokenParams &P, const Shared &S, const Lists &L, const Cta &cta, int d) {
    if (!S.good[d]) return;
    const float w = S.row[d].g * P.inv_hi, C = S.fix[d];
    for (int j = cta.lane; j < P.K; j += 32) {
        const int at = d * L.stride + j, id = L.ids[at], v = id / Kd::kPer;
        if (id >= 0 && v >= cta.slice0 && v < cta.slice0 + cta.slice_vecs)
            store_logit<Kd::DT>(P.grad + S.row[d].entry * P.grad_stride_bytes, id, w * (L.lp[at] - L.z[at] * C));
    }
}

// The divergence over the list's tokens and the rest, see include/specverify.h, as a sum of divergence_of's. Logarithms are pairs
// of floats up to their differences, and so is the normaliser: a small divergence or gradient is the difference of much larger
// terms.
template <class Kd>
__device__ __forceinline__ void finish_list(const TokenParams &P, Shared &S, const Lists &L, const Cta &cta, int d, const Part &p) {
    constexpr uint32_t all = 0xffffffffu;
    const Row &row = S.row[d];
    const long long e = row.entry;
    const int lane = cta.lane, K = P.K, kind = P.divergence;
    const float M = fmaxf(p.m, row.zmax);
    const bool bad = row.state == kBad || (row.state == kLive && (row.bad || p.n < 0 || M == -INFINITY));
    const bool good = row.state == kLive && !bad;
    const bool some = p.m > -INFINITY;  // the rest has mass
    if (row.state == kLive && bad && !row.bad && lane == 0 && cta.rank == 0) atomicOr(P.status, SPECVERIFY_STATUS_BAD_LOGIT);
    const bool early = !good || kind == SPECVERIFY_FKL || kind == SPECVERIFY_RKL;
    float loss = bad ? NAN : 0.0f, C = 0.0f;
    // the others' share of a gradient, (h_rest - q_rest C) / (s T) times 2^((z - m) c)
    auto known = [&](float d_rest) {  // (lane 1's)
        if (lane == 1) {
            const float f = some ? row.g * P.inv_hi * d_rest / p.s : 0.0f;
            S.coef[d] = bad ? make_float4(0.0f, NAN, 0.0f, 0.0f) : make_float4(some ? p.m : 0.0f, f, 0.0f, 0.0f);
            mbar_arrive(smem_u32(&S.known[d]));
        }
    };
    // The weights e^((z - M) / T) of the list's largest logit (even lanes) and of the rest's reference (odd lanes), and the
    // normaliser.
    float Zh = 1.0f, Zl = 0.0f;
    if (good) {
        float dh, dl, wh = 0.0f, wl = 0.0f, mh, ml;
        two_sum(lane & 1 ? p.m : row.zmax, -M, dh, dl);
        if (dh > P.far) {
            float xh, xl;
            over_T(P, dh, dl, xh, xl);
            ff_exp_pair(xh, xl, wh, wl);
        }
        ff_mul(wh, wl, lane & 1 ? p.s : row.zsum, lane & 1 ? 0.0f : row.zsum_l, mh, ml);
        ff_add(mh, ml, __shfl_xor_sync(all, mh, 1), __shfl_xor_sync(all, ml, 1), Zh, Zl);
        if (Kd::Grad && early) {
            // Here sum h is known without a look at the list: -sum p, and sum q ln(q / p) by the scout's sums. The stores need
            // not wait for the divergence (2.5 us for a list of 128). q of that logit and of the rest, and ln(q / p):
            float qh, ql;
            ff_div(lane & 1 ? mh : wh, lane & 1 ? ml : wl, Zh, Zl, qh, ql);
            if (kind == SPECVERIFY_FKL) {
                known(fmaf(qh, row.over, (qh - row.p_rest) + (ql - row.p_rest_l)));
            } else {
                const float ph = lane & 1 ? fmaxf(row.p_rest, 0x1p-20f) : row.p0, more = ((qh - ph) + (ql - (lane & 1 ? row.p_rest_l : row.p0_l))) / ph;
                const float t = fabsf(more) < 0.5f ? log1pf(more) : logf(qh) - (lane & 1 ? row.rest_h : row.lp0);
                const float part = qh > 0.0f ? lane & 1 ? qh * t : qh * fmaf(row.zsum, t, row.cross) : 0.0f;
                C = part + __shfl_xor_sync(all, part, 1);
                known(qh > 0.0f ? qh * (t - C) : 0.0f);
            }
        }
    } else if (Kd::Grad) {
        known(0.0f);
    }
    // the normaliser's logarithm; of q of the rest the logarithm, itself, and ln(p / q) of it
    float zh = 0.0f, zl = 0.0f, q_rest = 0.0f, r_rest = 0.0f;
    if (good) {
        float sh, sl, qh = -INFINITY, ql = 0.0f;
        ff_log_near(lane & 1 ? fmaxf(p.s, 0x1p-100f) : Zh, lane & 1 ? 0.0f : Zl, sh, sl);
        zh = __shfl_sync(all, sh, 0);
        zl = __shfl_sync(all, sl, 0);
        sh = __shfl_sync(all, sh, 1);
        sl = __shfl_sync(all, sl, 1);
        if (some) {
            ff_logprob(P, p.m, M, zh, zl, qh, ql);
            if (qh > -INFINITY) ff_add(qh, ql, sh, sl, qh, ql);
            q_rest = ff_exp(qh, ql);
        }
        r_rest = (row.rest_h - qh) + (row.rest_l - ql);
    }
    // h - q C where sum h = -sum p: q (1 + over) - p
    auto missing = [&](float pr, float q, float r) {
        return fmaf(q, row.over, fabsf(r) < 0.5f ? pr * expm1f(-r) : q - pr);
    };
    if (good) {
        float f = 0.0f, h = 0.0f, h_rest = 0.0f;
        // outcome K is the rest
        for (int j = lane; j <= K; j += 32) {
            const bool rest = j == K;
            const int at = d * L.stride + j;
            if (!rest && L.ids[at] < 0) continue;
            float q = q_rest, pr = row.p_rest, r = r_rest;  // r = ln(p / q)
            if (!rest) {
                float h, l;
                ff_logprob(P, L.z[at], M, zh, zl, h, l);
                q = ff_exp(h, l);
                pr = L.p[at];
                r = (L.lp[at] - h) - l;
            }
            float fj, hj;
            if (kind == SPECVERIFY_FKL) {
                fj = divergence_of(pr, q, r);
                hj = missing(pr, q, r);  // (with q C)
            } else if (kind == SPECVERIFY_RKL) {
                fj = divergence_of(q, rest ? fmaxf(pr, 0x1p-20f) : pr, -r);
                hj = q > 0.0f ? q * (-r - C) : 0.0f;  // (with q C)
            } else if (kind == SPECVERIFY_TVD) {
                const bool near = fabsf(r) < 0.5f;
                fj = 0.5f * fabsf(near ? pr * expm1f(-r) : pr - q);
                hj = 0.5f * q * ((near ? r < 0.0f : q > pr) ? 1.0f : (near ? r > 0.0f : q < pr) ? -1.0f : 0.0f);
            } else {
                // ln(m / q) = ln(1 + b (p / q - 1)), and the other way round; each has a p, a q that is 0 or neither
                const float b = P.beta, m = b * pr + (1.0f - b) * q;
                const float u = q > 0.0f ? ln_mixed(b, pr > 0.0f ? r : -INFINITY) : 0.0f;
                const float v = pr > 0.0f ? ln_mixed(1.0f - b, q > 0.0f ? -r : -INFINITY) : 0.0f;
                hj = -(1.0f - b) * q * u;
                fj = b * divergence_of(pr, m, -v) + (1.0f - b) * divergence_of(q, m, -u);
            }
            f += fj;
            h += hj;
            if (rest) {
                h_rest = hj;
            } else if (Kd::Grad) {
                L.lp[at] = hj;
                L.z[at] = q;
            }
        }
        loss = warp_sum(f);
        if (kind == SPECVERIFY_FKL) loss += row.over;
        if (kind == SPECVERIFY_RKL) loss -= row.over;
        if (Kd::Grad && early) C = 0.0f;
        if (Kd::Grad && !early) {
            C = warp_sum(h);
            known(__shfl_sync(all, h_rest, K & 31) - q_rest * C);
        }
    }
    if (lane == 0 && cta.rank == 0) P.loss[e] = loss;
    if (Kd::Grad && lane == 0) {
        S.fix[d] = C;
        S.good[d] = good;
    }
}

template <class Kd>
__device__ __forceinline__ void finish(const TokenParams &P, const Plan &plan, Shared &S, SharedTop *T, const Lists &L, const Cta &cta, int first) {
    int live = 0;
    for (int r = first;; r += Kd::kEpilogues) {
        const int d = cta.place(r);
        const uint32_t parity = cta.parity(r);
        if (!wait_bar(S.row_full[d], parity, S, P)) return;
        const int state = S.row[d].state;
        if (state == kEnd) return;
        Part p{-INFINITY, 0.0f, 0.0f, 0};
        if (!wait_bar(S.scouted[d], parity, S, P) || !wait_bar(S.summed[d], parity, S, P)) return;
        if (state == kLive && cta.cluster > 1) {
            if (!receive<Kd>(P, S, cta, live++, p)) return;
        } else if (state == kLive) {
            if (cta.lane < kConsumers) p = S.part[d][cta.lane];
            p = warp_fold<Kd>(P, p);
        }
        if (Kd::List) finish_list<Kd>(P, S, L, cta, d, p);
        else if (!finish_token<Kd>(P, plan, S, T, cta, d, p)) return;
        __syncwarp();
        if (Kd::Grad) {
            if (!wait_bar(S.stored[d], parity, S, P)) return;
            if (Kd::List) fix_list<Kd>(P, S, L, cta, d);
            else fix_token<Kd>(P, S, cta, d);
            __syncwarp();
        }
        if (cta.lane == 0) mbar_arrive(smem_u32(&S.row_free[d]));
    }
}

// ---------------------------------------------------------------------------

template <class Kd>
__global__ void __launch_bounds__(kThreads, 2) token_kernel(const __grid_constant__ TokenParams P, const __grid_constant__ Plan plan) {
    extern __shared__ __align__(128) uint8_t smem[];
    Shared &S = *reinterpret_cast<Shared *>(smem + (size_t)plan.slots * Kd::kChunkBytes);
    void *more = reinterpret_cast<uint8_t *>(&S) + (sizeof(Shared) + 15) / 16 * 16;
    SharedTop *top = Kd::Top ? static_cast<SharedTop *>(more) : nullptr;
    Lists list{};
    if (Kd::List) {
        list.stride = plan.list_stride;
        list.hash = static_cast<int32_t *>(more);
        list.ids = list.hash + kHash;
        list.z = reinterpret_cast<float *>(list.ids + kDepth * list.stride);
        list.lp = list.z + kDepth * list.stride;
        list.p = list.lp + kDepth * list.stride;
    }
    const int tid = threadIdx.x, warp = tid >> 5;

    Cta cta;
    cta.cluster = plan.cluster;
    cta.rank = plan.cluster > 1 ? (int)cluster_rank() : 0;
    cta.first = blockIdx.x / plan.cluster;
    const int vecs = (int)(((int64_t)P.V * Kd::kSize + 15) / 16), whole = P.V / Kd::kPer;
    cta.slice0 = min(vecs, cta.rank * plan.slice_vecs);
    cta.slice_vecs = min(vecs - cta.slice0, plan.slice_vecs);
    cta.chunks = (cta.slice_vecs + Kd::kChunkVecs - 1) / Kd::kChunkVecs;
    cta.whole_chunks = max(0, min(cta.slice_vecs, whole - cta.slice0)) / Kd::kChunkVecs;
    cta.lane = tid & 31;
    cta.depth_log = plan.depth_log;
    cta.ring = smem_u32(smem);
    cta.full = smem_u32(S.full);
    cta.ready = smem_u32(S.ready);
    cta.empty = smem_u32(S.empty);
    cta.words = reinterpret_cast<unsigned long long *>(smem + plan.words_at);

    if (tid == 0) {
        for (int i = 0; i < plan.slots; ++i) {
            mbar_init(smem_u32(&S.full[i]), 1);
            mbar_init(smem_u32(&S.ready[i]), 1);
            mbar_init(smem_u32(&S.empty[i]), kConsumers);
        }
        for (int i = 0; i < kDepth; ++i) {
            mbar_init(smem_u32(&S.row_full[i]), 1);
            mbar_init(smem_u32(&S.row_free[i]), kConsumers + (Kd::List ? 3 : 2));
            mbar_init(smem_u32(&S.sent[i]), 1);
            mbar_init(smem_u32(&S.summed[i]), kConsumers);
            mbar_init(smem_u32(&S.known[i]), 1);
            mbar_init(smem_u32(&S.stored[i]), kConsumers);
            mbar_init(smem_u32(&S.scouted[i]), 1);
            mbar_init(smem_u32(&S.bounded[i]), kConsumers);
        }
        mbar_init(smem_u32(&S.granted), 1);
        mbar_init(smem_u32(&S.acked), plan.cluster);
        mbar_init(smem_u32(&S.gathered), plan.cluster);
        S.asked = 0;
        S.abort = 0;
        if (Kd::Top)
            for (int i = 0; i < kTopDepth; ++i) top->found[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (Kd::List)
        for (int i = tid; i < kHash; i += kThreads) list.hash[i] = -1;
    if (plan.cluster > 1)
        for (int i = tid; i < 2 * plan.cluster * kConsumers * Kd::kWords; i += kThreads) cta.words[i] = 0;
    __syncthreads();
    if (plan.cluster > 1) cluster_sync();
    after_previous();

    Entries at{cta.first, 0, 0};
    if (warp < kConsumers) consume<Kd>(P, plan, S, top, cta);
    else if (warp == kScout) scout<Kd>(P, plan, S, list, cta, at);
    else if (warp == kProducer) produce<Kd>(P, plan, S, cta);
    else if (Kd::List && warp == kPatcher) patch<Kd>(P, plan, S, list, smem, cta);
    else if (warp == kEpilogue) finish<Kd>(P, plan, S, top, list, cta, 0);
    else if (Kd::kEpilogues == 2) finish<Kd>(P, plan, S, top, list, cta, 1);
    __syncwarp();
    // What other CTAs send may still be on its way here where somebody gave up.
    if (plan.cluster > 1) cluster_sync();
    if (!plan.dynamic) return;
    // The same of an answer to a request.
    if (warp == kScout) {
        int asked;
        asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(asked) : "r"(cluster_addr(&S.asked, 0)) : "memory");
        if (asked > at.answers) {
            if (asked > at.awaited && cta.lane == 0) mbar_arrive_expect_tx(smem_u32(&S.granted), 16);
            mbar_wait_bounded(smem_u32(&S.granted), (uint32_t)at.answers & 1u);
        }
    }
    if (plan.cluster > 1) cluster_sync();
}

// ---------------------------------------------------------------------------
// host

constexpr int kHalfSmem = 113 * 1024;  // of a CTA, two on an SM
constexpr int64_t kRereadBytes = 48 << 20;

// What fits the GPU of a kernel: clusters of 2^i CTAs at once.
template <class Kd>
struct Room {
    static inline int clusters[5];
};

// Rows over the GPU. One CTA a row where there are rows for every CTA that fits, else as many as do (a power of two). A
// gradient's rows go through L2 between their readings: no more of them at once than it holds well.
template <class Kd>
Plan make_plan(const TokenParams &P) {
    const int64_t vecs = ((int64_t)P.V * Kd::kSize + 15) / 16;
    Plan p{};
    p.depth_log = Kd::Top ? 1 : 2;
    p.list_stride = Kd::List ? (P.K + 31) / 32 * 32 : 0;
    const int fixed = (int)((sizeof(Shared) + 15) / 16 * 16) +
                      (Kd::List ? kHashBytes + p.list_stride * kListBytes : Kd::Top ? (int)((sizeof(SharedTop) + 15) / 16 * 16) : 0);
    const auto &room = Room<Kd>::clusters;
    int log = 0;
    if (Kd::Grad)
        while (log < 4 && (int64_t)room[log] * vecs * 16 > kRereadBytes) ++log;
    while (log < 4 && P.entries <= room[log + 1] && vecs >> log >= 256 && (!Kd::Top || P.k << (log + 1) <= kGathered)) ++log;
    p.cluster = 1 << log;
    p.slice_vecs = (int32_t)(((vecs + p.cluster - 1 >> log) + 31) / 32 * 32);
    const int words = log ? (2 * kConsumers * Kd::kWords * 8) << log : 0;
    p.slots = std::min(kMaxSlots, (kHalfSmem - fixed - words) / Kd::kChunkBytes);
    // (the sums of a cluster's rows have no way to keep one another apart: it has one row)
    p.dynamic = (Kd::Grad || log == 0) && P.entries <= INT32_MAX >> log;
    p.eager = vecs * 16 >> log <= p.slots * Kd::kChunkBytes;
    p.clusters = (int32_t)(p.dynamic ? P.entries : std::min<int64_t>(P.entries, std::max(1, room[log])));
    while (((((p.slice_vecs + Kd::kChunkVecs - 1) / Kd::kChunkVecs) + (1 << p.group_log) - 1) >> p.group_log) > kGroupRows) ++p.group_log;
    p.words_at = p.slots * Kd::kChunkBytes + fixed;
    p.smem = p.words_at + words;
    return p;
}

template <class Kd>
cudaError_t launch(const TokenParams &P, cudaStream_t s) {
    const Plan plan = make_plan<Kd>(P);
    return launch_after(token_kernel<Kd>, dim3((unsigned)(plan.clusters * plan.cluster)), kThreads, plan.smem, s, plan.cluster, P,
                        plan);
}

template <class Kd>
cudaError_t prepare() {
    cudaError_t e = cudaFuncSetAttribute(token_kernel<Kd>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHalfSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(token_kernel<Kd>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    for (int log = 0; log < 5 && e == cudaSuccess; ++log) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1u << log;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(1u << log);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kHalfSmem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&Room<Kd>::clusters[log], token_kernel<Kd>, &cfg);
    }
    return e;
}

}  // namespace

}  // namespace sv
