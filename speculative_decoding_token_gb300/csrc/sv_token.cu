// sv_token.cu -- log-probabilities of given tokens (with entropy, rank and top
// alternatives), the divergence of a draft's rows from its target's top tokens,
// and the gradients of both: one pass over rows of logits.
//
// A row is taken by a cluster of S CTAs, each a slice of it; S = 1 where there
// are rows enough. Slices come in chunks of 8 KiB by bulk copies into a ring of
// shared memory. The warps of a CTA:
//   consumers (8)  a chunk's vectors, two a thread: the running maximum m, the
//                  sum s of 2^((z - m) c) and t of 2^((z - m) c) (z - m), c =
//                  log2(e) / T; for a gradient, once the row's sums are known,
//                  again over the same chunks, to store it;
//   scout          what a row's entry asks for (its token, or its list with
//                  the logits and probabilities of it), up to kDepth rows ahead;
//   producer       the copies;
//   patcher        (lists) takes the listed tokens out of a chunk that has
//                  arrived (-inf), so that the sums are over the rest alone;
//   epilogue       merges the warps' sums (and the cluster's), picks the top
//                  tokens, writes the results, and hands the consumers what a
//                  gradient's second reading needs.
// No warp waits for the end of a row but the consumers of a gradient.
#include "sv_token.h"
#include "sv_rows.cuh"
#include "sv_tree.h"

#include <algorithm>

namespace sv {

namespace token {

constexpr int kConsumers = 8;                     // warps
constexpr int kScout = kConsumers, kProducer = kScout + 1, kPatcher = kProducer + 1, kEpilogue = kPatcher + 1;
constexpr int kThreads = (kEpilogue + 1) * 32;
constexpr int kVecs = 2;                          // 16-byte vectors of a chunk that a thread takes
constexpr int kChunkVecs = kConsumers * 32 * kVecs;
constexpr int kChunkBytes = kChunkVecs * 16;
constexpr int kMaxSlots = 26;
constexpr int kDepth = 4;                         // rows between the scout and the epilogue at most
constexpr int kTopDepth = 2;                      // the same where top tokens are asked for (their buffers are large)
constexpr int kMaxCluster = 16;
constexpr int kCandidates = kChunkVecs + 128;     // vectors that may hold top tokens: a chunk of ties, and more
constexpr int kKeys = 1024;                       // tokens among them
constexpr int kGathered = 512;                    // keys that a cluster's CTAs send to its first
constexpr int kHash = 1024;

enum State { kLive = 0, kSkip = 1, kBad = 2 };

// What the scout knows of a row.
struct Row {
    const char *z;
    long long entry;
    int state;
    int y;
    float zy;
    float p_rest;  // of a list: what it leaves of one
    float g, h;    // what the gradient is multiplied by
};

// Sums over part of a row: s and t relative to m (see above); n tokens before
// the given one, -1: a bad logit.
struct Part {
    float m, s, t;
    int n;
};

struct Shared {
    uint64_t full[kMaxSlots], ready[kMaxSlots], empty[kMaxSlots];
    uint64_t row_full[kDepth], row_free[kDepth], summed[kDepth], known[kDepth], stored[kDepth], bounded[kDepth];
    uint64_t exchanged[2];
    Row row[kDepth];
    Part part[kDepth][kConsumers];
    Part others[2][kMaxCluster];
    float4 coef[kDepth];  // of the gradient: reference, factor, slope
    int32_t abort;
};

// Top tokens: a key is a logit's bits, made to order as it does, over its
// token's, inverted: keys fall in the order of alternatives, and 0 is none.
struct SharedTop {
    unsigned long long bound[kTopDepth][kConsumers];  // that many tokens are at least so large; chunk
    uint4 vec[kTopDepth][kCandidates];
    int32_t at[kTopDepth][kCandidates];
    unsigned long long keys[kKeys];
    unsigned long long best[kMaxAlternatives];
    unsigned long long gathered[kGathered];
    unsigned count[kTopDepth];
};

struct SharedList {
    int32_t ids[kDepth][kMaxList];
    float z[kDepth][kMaxList];
    float lp[kDepth][kMaxList];  // the target's log-probability
    int32_t hash[kHash];
};

// How a call's rows are laid out over the GPU.
struct Plan {
    int32_t cluster;      // CTAs of a row
    int32_t slots;        // of a ring
    int32_t slice_vecs;   // vectors of a slice, but the last's
    int32_t lag;          // rows between the two readings of a gradient
    int32_t depth_log;    // rows between the scout and the epilogue
    int32_t clusters;
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

template <int DT>
struct Type {
    static constexpr int kSize = DT == SV_DT_FP32 ? 4 : 2;
    static constexpr int kPer = 16 / kSize;  // logits of a vector
    static constexpr uint32_t kNegInf = DT == SV_DT_FP32 ? 0xff800000u : 0xff80ff80u;
};

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

// The least exponent argument that is told from -inf: a weight of 0 either way,
// and its product with the argument is 0 and not NaN.
constexpr float kFar = -0x1p100f;

__device__ __forceinline__ void merge(Part &a, const Part &b, float c) {
    a.n = a.n < 0 || b.n < 0 ? -1 : a.n + b.n;
    if (b.m == -INFINITY) return;
    if (a.m == -INFINITY) {
        a.m = b.m;
        a.s = b.s;
        a.t = b.t;
        return;
    }
    const float m = fmaxf(a.m, b.m);
    const float da = fmaxf(a.m - m, kFar), db = fmaxf(b.m - m, kFar);
    const float fa = ex2_approx(da * c), fb = ex2_approx(db * c);
    a.t = fa * fmaf(da, a.s, a.t) + fb * fmaf(db, b.s, b.t);
    a.s = fa * a.s + fb * b.s;
    a.m = m;
}

__device__ __forceinline__ Part warp_merge(Part a, float c) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        Part b;
        b.m = __shfl_xor_sync(0xffffffffu, a.m, off);
        b.s = __shfl_xor_sync(0xffffffffu, a.s, off);
        b.t = __shfl_xor_sync(0xffffffffu, a.t, off);
        b.n = __shfl_xor_sync(0xffffffffu, a.n, off);
        merge(a, b, c);
    }
    return a;
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

// wait_on for what other CTAs of the cluster have sent
__device__ __forceinline__ bool wait_on_cluster(uint64_t &bar, uint32_t parity, int32_t &abort, int32_t *status,
                                                uint64_t limit) {
    if (!wait_on(bar, parity, abort, status, limit)) return false;
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    return true;
}

// A CTA's view of the call.
struct Cta {
    int rank, cluster;
    long long first, step;   // entries
    int slice0, slice_vecs;  // vectors of the row
    int chunks;
    int lane;
    int depth_log;

    __device__ __forceinline__ int place(int r) const { return r & ((1 << depth_log) - 1); }
    __device__ __forceinline__ uint32_t parity(int r) const { return (uint32_t)r >> depth_log & 1u; }
};

// ---------------------------------------------------------------------------
// consumers

// The sums of a row's slice, vectors of chunk after chunk. G: its chunks stay for the gradient.
template <int DT, bool LIST, bool G>
__device__ __forceinline__ bool sum_slice(const TokenParams &P, const Plan &plan, Shared &S, SharedTop *top, const uint8_t *ring,
                                          const Cta &cta, int d, uint32_t row_parity, int &slot, uint32_t &phase) {
    using Ty = Type<DT>;
    const int tid = threadIdx.x, lane = cta.lane, warp = tid >> 5;
    const Row &row = S.row[d];
    const bool ent = !LIST && (P.entropy || P.g_entropy);
    const bool rank = !LIST && !G && P.rank;
    const int k = LIST || G ? 0 : P.k;
    const int nth = (k + kConsumers - 1) / kConsumers;
    const int whole = P.V / Ty::kPer, rest = P.V - whole * Ty::kPer;
    float m = -INFINITY;
    f32x2 s0 = 0ull, s1 = 0ull, t0 = 0ull, t1 = 0ull;
    bool bad = false;
    int before = 0;
    uint32_t bound = 0;     // order bits that a vector has to reach
    int bound_chunk = 0;    // and pass, in later chunks than this one
    const f32x2 c2 = pack2(P.c, P.c);
    for (int i = 0; i < cta.chunks; ++i) {
        if (!wait_on(S.full[slot], phase, S.abort, P.status, P.wait_ns)) return false;
        if (LIST && !wait_on(S.ready[slot], phase, S.abort, P.status, P.wait_ns)) return false;
        const uint4 *chunk = reinterpret_cast<const uint4 *>(ring + (size_t)slot * kChunkBytes);
        const int n = min(kChunkVecs, cta.slice_vecs - i * kChunkVecs);
        const int v0 = cta.slice0 + i * kChunkVecs;  // of the row
        uint4 w[kVecs];
        float vm[kVecs];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int v = tid + j * kConsumers * 32;
            if (v < n) w[j] = chunk[v];
            else w[j] = make_uint4(Ty::kNegInf, Ty::kNegInf, Ty::kNegInf, Ty::kNegInf);
            if (!LIST && rest && v < n && v0 + v == whole) {  // the ragged end of the row, which no copy brings
                uint32_t x[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    x[q] = Ty::kNegInf;
#pragma unroll
                    for (int e = 0; e < 4 / Ty::kSize; ++e) {
                        const int at = q * (4 / Ty::kSize) + e;
                        if (at >= rest) continue;
                        const char *p = row.z + ((int64_t)whole * Ty::kPer + at) * Ty::kSize;
                        if (DT == SV_DT_FP32) x[q] = *reinterpret_cast<const volatile uint32_t *>(p);
                        else x[q] = (x[q] & ~(0xffffu << (16 * e))) |
                                    (uint32_t)*reinterpret_cast<const volatile uint16_t *>(p) << (16 * e);
                    }
                }
                w[j] = make_uint4(x[0], x[1], x[2], x[3]);
            }
        }
        if (!G) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.empty[slot]));
        }
        if (++slot == plan.slots) {
            slot = 0;
            phase ^= 1u;
        }
        float cm = -INFINITY;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            vm[j] = vec_max<DT>(w[j]);
            cm = max_nan(cm, vm[j]);
        }
        if (!(cm < INFINITY)) {
            bad = true;
            cm = -INFINITY;
        }
        if (cm > m) {
            if (m != -INFINITY) {
                const float dm = fmaxf(m - cm, kFar), f = ex2_approx(dm * P.c);
                const f32x2 f2 = pack2(f, f), d2 = pack2(dm, dm);
                if (ent) {
                    t0 = mul2(f2, fma2(d2, s0, t0));
                    t1 = mul2(f2, fma2(d2, s1, t1));
                }
                s0 = mul2(f2, s0);
                s1 = mul2(f2, s1);
            }
            m = cm;
        }
        if (m != -INFINITY) {
            const f32x2 nm = pack2(-m, -m);
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
#pragma unroll
                for (int q = 0; q < Ty::kPer / 2; ++q) {
                    const float2 z = pair_of<DT>(w[j], q);
                    float2 dz = unpack2(add2(pack2(z.x, z.y), nm));
                    if (ent) {
                        dz.x = fmaxf(dz.x, kFar);
                        dz.y = fmaxf(dz.y, kFar);
                    }
                    const f32x2 d2 = pack2(dz.x, dz.y);
                    const float2 x = unpack2(mul2(d2, c2));
                    const f32x2 e2 = pack2(ex2_approx(x.x), ex2_approx(x.y));
                    if (q & 1) {
                        s1 = add2(s1, e2);
                        if (ent) t1 = fma2(e2, d2, t1);
                    } else {
                        s0 = add2(s0, e2);
                        if (ent) t0 = fma2(e2, d2, t0);
                    }
                }
        }
        if (rank) {
            const float zy = row.zy;
            const int y = row.y;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int v = tid + j * kConsumers * 32;
                // the indexes of what fills a short chunk belong to the next slice
                const int e0 = v < n ? (v0 + v) * Ty::kPer : P.V;
#pragma unroll
                for (int q = 0; q < Ty::kPer / 2; ++q) {
                    const float2 z = pair_of<DT>(w[j], q);
                    before += (z.x > zy || (z.x == zy && e0 + 2 * q < y)) ? 1 : 0;
                    before += (z.y > zy || (z.y == zy && e0 + 2 * q + 1 < y)) ? 1 : 0;
                }
            }
        }
        if (k > 0) {
            // Each warp bounds the k-th largest logit by the nth largest of its lanes' maxima: 8 warps have 8 nth >= k
            // tokens that large. The bound of the first chunk is everybody's; it then rises at chunks 1, 3, 7, ...
            const bool last = i + 1 == cta.chunks;
            if ((i & (i + 1)) == 0 || last) {
                const uint32_t mine = warp_nth(order_bits(m), nth, lane);
                if (lane == 0)
                    *(volatile unsigned long long *)&top->bound[d][warp] = ((unsigned long long)mine << 32) | (uint32_t)i;
                if (i == 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&S.bounded[d]));
                    if (!wait_on(S.bounded[d], row_parity, S.abort, P.status, P.wait_ns)) return false;
                }
            }
            if ((i & (i - 1)) == 0) {
                const unsigned long long b = lane < kConsumers ? *(volatile unsigned long long *)&top->bound[d][lane] : ~0ull << 32;
                bound = __reduce_min_sync(0xffffffffu, (uint32_t)(b >> 32));
                bound_chunk = (int)__reduce_max_sync(0xffffffffu, (uint32_t)b);
            }
            // Tokens that equal the bound come after the ones that made it, once these lie in earlier chunks.
            const float least = from_order_bits(bound);
            const bool strict = i > bound_chunk;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int v = tid + j * kConsumers * 32;
                if (v < n && (strict ? vm[j] > least : vm[j] >= least)) {
                    const unsigned at = atomicAdd(&top->count[d], 1u);
                    if (at < kCandidates) {
                        top->vec[d][at] = w[j];
                        top->at[d][at] = v0 + v;
                    }
                }
            }
        }
    }
    if (k > 0 && cta.chunks == 0 && lane == 0) mbar_arrive(smem_u32(&S.bounded[d]));
    const float2 a = unpack2(s0), b = unpack2(s1), e = unpack2(t0), f = unpack2(t1);
    Part p{m, (a.x + a.y) + (b.x + b.y), (e.x + e.y) + (f.x + f.y), bad ? -1 : before};
    p = warp_merge(p, P.c);
    if (lane == 0) {
        S.part[d][warp] = p;
        mbar_arrive(smem_u32(&S.summed[d]));
    }
    return true;
}

// The gradient of a row's slice.
template <int DT, bool LIST>
__device__ __forceinline__ bool store_slice(const TokenParams &P, const Plan &plan, Shared &S, const uint8_t *ring, const Cta &cta,
                                            int d, uint32_t row_parity, int &slot) {
    using Ty = Type<DT>;
    const int tid = threadIdx.x, lane = cta.lane;
    const int whole = P.V / Ty::kPer, rest = P.V - whole * Ty::kPer;
    const int state = S.row[d].state;
    char *out = P.grad + S.row[d].entry * P.grad_stride_bytes;
    float4 cf = make_float4(0.0f, state == kBad ? NAN : 0.0f, 0.0f, 0.0f);
    if (state == kLive) {
        if (!wait_on(S.known[d], row_parity, S.abort, P.status, P.wait_ns)) return false;
        cf = S.coef[d];
    }
    const bool ent = !LIST && P.g_entropy;
    const f32x2 nm = pack2(-cf.x, -cf.x), c2 = pack2(P.c, P.c), a2 = pack2(cf.y, cf.y), b2 = pack2(cf.z, cf.z);
    for (int i = 0; i < cta.chunks; ++i) {
        const uint4 *chunk = reinterpret_cast<const uint4 *>(ring + (size_t)slot * kChunkBytes);
        const int n = min(kChunkVecs, cta.slice_vecs - i * kChunkVecs);
        const int v0 = cta.slice0 + i * kChunkVecs;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int v = tid + j * kConsumers * 32;
            if (v >= n) continue;
            float g[Ty::kPer];
            if (state == kLive) {
                uint4 w = chunk[v];
                if (!LIST && rest && v0 + v == whole) {
                    uint32_t x[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int q = 0; q < Ty::kPer; ++q) {
                        if (q >= rest) continue;
                        const char *p = S.row[d].z + ((int64_t)whole * Ty::kPer + q) * Ty::kSize;
                        if (DT == SV_DT_FP32) x[q & 3] = *reinterpret_cast<const volatile uint32_t *>(p);
                        else x[(q >> 1) & 3] |= (uint32_t)*reinterpret_cast<const volatile uint16_t *>(p) << (16 * (q & 1));
                    }
                    w = make_uint4(x[0], x[1], x[2], x[3]);
                }
#pragma unroll
                for (int q = 0; q < Ty::kPer / 2; ++q) {
                    const float2 z = pair_of<DT>(w, q);
                    float2 dz = unpack2(add2(pack2(z.x, z.y), nm));
                    if (ent) {
                        dz.x = fmaxf(dz.x, kFar);
                        dz.y = fmaxf(dz.y, kFar);
                    }
                    const f32x2 d2 = pack2(dz.x, dz.y);
                    const float2 x = unpack2(mul2(d2, c2));
                    const f32x2 e2 = pack2(ex2_approx(x.x), ex2_approx(x.y));
                    const float2 r = unpack2(mul2(e2, ent ? fma2(b2, d2, a2) : a2));
                    g[2 * q] = r.x;
                    g[2 * q + 1] = r.y;
                }
            } else {
#pragma unroll
                for (int q = 0; q < Ty::kPer; ++q) g[q] = cf.y;
            }
            char *to = out + (int64_t)(v0 + v) * 16;
            if (v0 + v < whole) {
                uint4 r;
                if (DT == SV_DT_FP32)
                    r = make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3]));
                else
                    r = make_uint4(to_bf16x2(g[0], g[1]), to_bf16x2(g[2], g[3]), to_bf16x2(g[4 % Ty::kPer], g[5 % Ty::kPer]),
                                   to_bf16x2(g[6 % Ty::kPer], g[7 % Ty::kPer]));
                *reinterpret_cast<uint4 *>(to) = r;
            } else {
#pragma unroll
                for (int q = 0; q < Ty::kPer; ++q)
                    if (q < rest) store_logit<DT>(to, q, g[q]);
            }
        }
        if (state == kLive) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&S.empty[slot]));
            if (++slot == plan.slots) slot = 0;
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&S.stored[d]));
    return true;
}

template <int DT, bool LIST, bool G>
__device__ __forceinline__ void consume(const TokenParams &P, const Plan &plan, Shared &S, SharedTop *top, const uint8_t *ring,
                                        const Cta &cta) {
    int slot = 0, gslot = 0, r = 0;
    uint32_t phase = 0;
    auto store = [&](int g) {
        const int d = cta.place(g);
        if (!store_slice<DT, LIST>(P, plan, S, ring, cta, d, cta.parity(g), gslot)) return false;
        if (cta.lane == 0) mbar_arrive(smem_u32(&S.row_free[d]));
        return true;
    };
    for (long long e = cta.first; e < P.entries; e += cta.step, ++r) {
        const int d = cta.place(r);
        if (!wait_on(S.row_full[d], cta.parity(r), S.abort, P.status, P.wait_ns)) return;
        if (S.row[d].state == kLive) {
            if (!sum_slice<DT, LIST, G>(P, plan, S, top, ring, cta, d, cta.parity(r), slot, phase)) return;
        } else if (cta.lane == 0) {
            if (top) mbar_arrive(smem_u32(&S.bounded[d]));
            mbar_arrive(smem_u32(&S.summed[d]));
        }
        if (!G) {
            __syncwarp();
            if (cta.lane == 0) mbar_arrive(smem_u32(&S.row_free[d]));
        } else if (r >= plan.lag && !store(r - plan.lag)) {
            return;
        }
    }
    if (G && plan.lag && r > 0) store(r - 1);
}

// ---------------------------------------------------------------------------
// scout

template <int DT>
__device__ __forceinline__ void scout_token(const TokenParams &P, Row &row, long long e) {
    const int y = P.tokens[e];
    int64_t r = e;
    int bits = 0;
    if (y != -1) {
        if (P.row_off) r = P.row_off[e / P.M] + (P.path ? (int64_t)P.path[e] : (int64_t)(e % P.M));
        if (y < 0 || y >= P.V) bits = SPECVERIFY_STATUS_BAD_TOKEN;
        else if (r < 0 || r >= P.rows) bits = SPECVERIFY_STATUS_BAD_ROW;
    }
    row.z = P.logits + r * P.stride_bytes;
    row.entry = e;
    row.y = y;
    row.state = y == -1 ? kSkip : bits ? kBad : kLive;
    row.zy = row.state == kLive ? plain_logit<DT>(row.z, y) : 0.0f;
    if (P.grad) {
        row.g = P.g_logprob[e];
        row.h = P.g_entropy ? P.g_entropy[e] : 0.0f;
    }
    if (bits) atomicOr(P.status, bits);
}

// A list: its ids, the draft's logits of them, the target's log-probabilities.
template <int DT>
__device__ void scout_list(const TokenParams &P, Row &row, SharedList &L, int d, long long e, int lane) {
    constexpr uint32_t all = 0xffffffffu;
    const char *z = P.logits + e * P.stride_bytes;
    int bits = 0;
    bool any = false;
    float top = -INFINITY;
    for (int j = lane; j < P.K; j += 32) {
        int id = P.ids[e * P.K + j];
        float zk = -INFINITY, t = -INFINITY;
        if (id < -1 || id >= P.V) {
            bits |= SPECVERIFY_STATUS_BAD_TOKEN;
            id = -1;
        } else if (id >= 0) {
            any = true;
            zk = plain_logit<DT>(z, id);
            t = P.target_bf16 ? plain_logit<SV_DT_BF16>(P.target, e * P.K + j) : plain_logit<SV_DT_FP32>(P.target, e * P.K + j);
            if (!(zk < INFINITY) || !(t < INFINITY)) bits |= SPECVERIFY_STATUS_BAD_LOGIT;
            // twice the same id: one of its entries finds the other in the table
            uint32_t at = (uint32_t)id * 2654435761u >> 22;
            for (int tries = 0; tries < kHash; ++tries, at = (at + 1) % kHash) {
                const int was = atomicCAS(&L.hash[at], -1, id);
                if (was == id) bits |= SPECVERIFY_STATUS_BAD_TOKEN;
                if (was == -1 || was == id) break;
            }
        }
        L.ids[d][j] = id;
        L.z[d][j] = zk;
        L.lp[d][j] = t;
        top = fmaxf(top, t);
    }
    __syncwarp();
    for (int j = lane; j < kHash / 4; j += 32) reinterpret_cast<int4 *>(L.hash)[j] = make_int4(-1, -1, -1, -1);
    bits = __reduce_or_sync(all, bits);
    any = __any_sync(all, any);
    float p_rest = 0.0f;
    if (!bits && any) {
        if (P.form == SPECVERIFY_TARGET_LOGITS) {
            top = warp_max(top);
            float sum = 0.0f, lh = 0.0f, ll = 0.0f;
            for (int j = lane; j < P.K; j += 32) {
                float h, l;
                ff_logprob(P, L.lp[d][j], top, 0.0f, 0.0f, h, l);
                sum += L.lp[d][j] == -INFINITY ? 0.0f : ff_exp(h, l);
            }
            sum = warp_sum(sum);
            if (top == -INFINITY) bits = SPECVERIFY_STATUS_BAD_LOGIT;  // a target of nothing
            else ff_log(sum, lh, ll);
            for (int j = lane; j < P.K; j += 32) {
                float h, l;
                ff_logprob(P, L.lp[d][j], top, lh, ll, h, l);
                L.lp[d][j] = L.lp[d][j] == -INFINITY ? -INFINITY : h;
            }
        } else {
            // One less a sum close to it: in 64 bits, or little would be left of it. (Off everybody's way: the scout is rows
            // ahead.)
            double sum = 0.0;
            for (int j = lane; j < P.K; j += 32)
                if (L.lp[d][j] > -INFINITY) sum += exp((double)L.lp[d][j]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(all, sum, off);
            p_rest = (float)fmax(1.0 - sum, 0.0);
        }
    }
    if (lane == 0) {
        row.z = z;
        row.entry = e;
        row.state = bits ? kBad : any ? kLive : kSkip;
        row.p_rest = p_rest;
        row.g = P.weight ? P.weight[e] : 1.0f;
        if (bits) atomicOr(P.status, bits);
    }
}

template <int DT, bool LIST>
__device__ __forceinline__ void scout(const TokenParams &P, Shared &S, SharedTop *top, SharedList *list, const Cta &cta) {
    int r = 0;
    for (long long e = cta.first; e < P.entries; e += cta.step, ++r) {
        const int d = cta.place(r);
        if (!wait_on(S.row_free[d], cta.parity(r) ^ 1u, S.abort, P.status, P.wait_ns)) return;
        if (LIST) {
            scout_list<DT>(P, S.row[d], *list, d, e, cta.lane);
        } else if (cta.lane == 0) {
            scout_token<DT>(P, S.row[d], e);
            if (top) top->count[d] = 0;
        }
        __syncwarp();
        if (cta.lane == 0) mbar_arrive(smem_u32(&S.row_full[d]));
    }
}

// ---------------------------------------------------------------------------
// producer and patcher

template <int DT>
__device__ __forceinline__ void produce(const TokenParams &P, const Plan &plan, Shared &S, uint8_t *ring, const Cta &cta) {
    const int64_t row_bytes = (int64_t)P.V * Type<DT>::kSize & ~15ll;
    int slot = 0, r = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    for (long long e = cta.first; e < P.entries && ok; e += cta.step, ++r) {
        const int d = cta.place(r);
        ok = wait_on(S.row_full[d], cta.parity(r), S.abort, P.status, P.wait_ns);
        if (!ok) break;
        const char *z = S.row[d].z;
        const bool live = S.row[d].state == kLive;
        __syncwarp();
        if (cta.lane == 0) mbar_arrive(smem_u32(&S.row_free[d]));
        if (!live) continue;
        for (int i = 0; i < cta.chunks && ok; ++i) {
            ok = wait_on(S.empty[slot], phase ^ 1u, S.abort, P.status, P.wait_ns);
            if (!ok) break;
            if (cta.lane == 0) {
                const int64_t off = ((int64_t)cta.slice0 + (int64_t)i * kChunkVecs) * 16;
                const int n = min(kChunkVecs, cta.slice_vecs - i * kChunkVecs) * 16;
                const int bytes = (int)min((int64_t)n, row_bytes - off);
                const uint32_t bar = smem_u32(&S.full[slot]);
                if (bytes > 0) {
                    mbar_arrive_expect_tx(bar, (uint32_t)bytes);
                    bulk_load(smem_u32(ring + (size_t)slot * kChunkBytes), z + off, (uint32_t)bytes, bar);
                } else {
                    mbar_arrive(bar);
                }
            }
            ++issued;
            if (++slot == plan.slots) {
                slot = 0;
                phase ^= 1u;
            }
        }
    }
    // no copy outlives its CTA, also where those who needed it gave up
    for (long long u = max(0ll, issued - plan.slots); u < issued; ++u)
        mbar_wait_bounded(smem_u32(&S.full[u % plan.slots]), u / plan.slots & 1);
}

template <int DT>
__device__ __forceinline__ void patch(const TokenParams &P, const Plan &plan, Shared &S, const SharedList &L, uint8_t *ring,
                                      const Cta &cta) {
    using Ty = Type<DT>;
    const int whole = P.V / Ty::kPer, rest = P.V - whole * Ty::kPer;
    int slot = 0, r = 0;
    uint32_t phase = 0;
    for (long long e = cta.first; e < P.entries; e += cta.step, ++r) {
        const int d = cta.place(r);
        if (!wait_on(S.row_full[d], cta.parity(r), S.abort, P.status, P.wait_ns)) return;
        for (int i = 0; i < (S.row[d].state == kLive ? cta.chunks : 0); ++i) {
            if (!wait_on(S.full[slot], phase, S.abort, P.status, P.wait_ns)) return;
            uint8_t *chunk = ring + (size_t)slot * kChunkBytes;
            const int v0 = cta.slice0 + i * kChunkVecs;
            const int n = min(kChunkVecs, cta.slice_vecs - i * kChunkVecs);
            if (rest && v0 <= whole && whole < v0 + n) {  // the ragged end of the row, which no copy brings
                if (cta.lane < Ty::kPer) {
                    const float x = cta.lane < rest ? plain_logit<DT>(S.row[d].z, (int64_t)whole * Ty::kPer + cta.lane) : -INFINITY;
                    store_logit<DT>(reinterpret_cast<char *>(chunk + (whole - v0) * 16), cta.lane, x);
                }
                __syncwarp();
            }
            for (int j = cta.lane; j < P.K; j += 32) {
                const int at = L.ids[d][j] - v0 * Ty::kPer;
                if (at >= 0 && at < n * Ty::kPer) store_logit<DT>(reinterpret_cast<char *>(chunk), at, -INFINITY);
            }
            // the next copy into this slot comes after these stores
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (cta.lane == 0) mbar_arrive(smem_u32(&S.ready[slot]));
            if (++slot == plan.slots) {
                slot = 0;
                phase ^= 1u;
            }
        }
        __syncwarp();
        if (cta.lane == 0) mbar_arrive(smem_u32(&S.row_free[d]));
    }
}

// ---------------------------------------------------------------------------
// epilogue

// Calls f with the keys of the n candidates' tokens, or (n < 0) of the whole slice, read once more from memory.
template <int DT, class F>
__device__ __forceinline__ void each_key(const TokenParams &P, const Row &row, const SharedTop &T, int d, int n, const Cta &cta, F &&f) {
    using Ty = Type<DT>;
    auto vector = [&](const uint4 &w, int at) {
        float x[Ty::kPer];
        vec_floats<DT>(w, x);
#pragma unroll
        for (int q = 0; q < Ty::kPer; ++q)
            if (at * Ty::kPer + q < P.V) f(order_key(x[q], at * Ty::kPer + q));
    };
    if (n >= 0) {
        for (int i = cta.lane; i < n; i += 32) vector(T.vec[d][i], T.at[d][i]);
        return;
    }
    const int whole = P.V / Ty::kPer, end = min(whole, cta.slice0 + cta.slice_vecs);
    const uint4 *z = reinterpret_cast<const uint4 *>(row.z);
    for (int v = cta.slice0 + cta.lane; v < end; v += 128) {
        uint4 w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (v + 32 * q < end) w[q] = __ldg(z + v + 32 * q);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (v + 32 * q < end) vector(w[q], v + 32 * q);
    }
    const int at = whole * Ty::kPer + cta.lane;  // the ragged end
    if (cta.slice0 + cta.slice_vecs > whole && at < P.V) f(order_key(load_logit<DT>(row.z, at), at));
}

// The k best keys of the CTA's slice, in order, in T.best (0 where there are none).
template <int DT>
__device__ void select_top(const TokenParams &P, const Row &row, SharedTop &T, int d, const Cta &cta) {
    constexpr uint32_t all = 0xffffffffu;
    const int lane = cta.lane, k = P.k;
    const unsigned found = *(volatile unsigned *)&T.count[d];
    int n = found <= kCandidates ? (int)found : -1;
    // the last bound: k tokens are at least so large, or there are not that many
    const unsigned long long b = lane < kConsumers ? T.bound[d][lane] : ~0ull;
    unsigned long long least = (unsigned long long)__reduce_min_sync(all, (uint32_t)(b >> 32)) << 32;
    if (cta.chunks == 0) {
        least = 0;
        n = 0;
    }
    auto count = [&](unsigned long long key) {
        int c = 0;
        each_key<DT>(P, row, T, d, n, cta, [&](unsigned long long x) { c += x >= key ? 1 : 0; });
        return (int)__reduce_add_sync(all, (unsigned)c);
    };
    // More than fit (many equal logits, or rows that rise): the largest key that k tokens reach, a bit at a time.
    if (count(least) > kKeys) {
        unsigned long long key = 0;
        for (int bit = 63; bit >= 0; --bit)
            if (count(key | 1ull << bit) >= k) key |= 1ull << bit;
        least = max(least, key);
    }
    int m = 0;
    {
        // keys into one list, each lane's behind those of the lanes before it
        int mine = 0;
        each_key<DT>(P, row, T, d, n, cta, [&](unsigned long long x) { mine += x >= least ? 1 : 0; });
        int incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(all, incl, off);
            if (lane >= off) incl += y;
        }
        m = __shfl_sync(all, incl, 31);
        int at = incl - mine;
        each_key<DT>(P, row, T, d, n, cta, [&](unsigned long long x) {
            if (x >= least) T.keys[at++] = x;
        });
    }
    for (int i = lane; i < k; i += 32) T.best[i] = 0;
    __syncwarp();
    // a key's place is the number of larger ones
    for (int i0 = 0; i0 < m; i0 += 128) {
        unsigned long long x[4];
        int place[4] = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = i0 + 32 * q + lane < m ? T.keys[i0 + 32 * q + lane] : 0;
        for (int i = 0; i < m; ++i) {
            const unsigned long long o = T.keys[i];
#pragma unroll
            for (int q = 0; q < 4; ++q) place[q] += o > x[q] ? 1 : 0;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (x[q] && place[q] < k) T.best[place[q]] = x[q];
    }
    __syncwarp();
}

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

// The cluster's sums from each CTA's. Rows of a gradient follow one another through two sets of slots: a CTA sends a row's
// sums once it has read those of the row before, so a slot is free again when its next sums arrive.
__device__ __forceinline__ bool exchange(const TokenParams &P, Shared &S, const Cta &cta, int x, Part &p) {
    const int lane = cta.lane, set = x & 1;
    if (lane < cta.cluster) {
        st_cluster_f4(cluster_addr(&S.others[set][cta.rank], lane), make_float4(p.m, p.s, p.t, __int_as_float(p.n)));
        cluster_arrive(S.exchanged[set], lane);
    }
    if (!wait_on_cluster(S.exchanged[set], x >> 1 & 1, S.abort, P.status, P.wait_ns)) return false;
    p = lane < cta.cluster ? S.others[set][lane] : Part{-INFINITY, 0.0f, 0.0f, 0};
    p = warp_merge(p, P.c);
    return true;
}

template <int DT, bool G>
__device__ __forceinline__ bool finish_token(const TokenParams &P, Shared &S, SharedTop *T, const Cta &cta, int d, uint32_t parity,
                                             Part p, int &x) {
    const Row &row = S.row[d];
    const long long e = row.entry;
    const int lane = cta.lane, k = G ? 0 : P.k;
    const bool alone = cta.cluster == 1;
    if (row.state == kLive) {
        if (k) {
            select_top<DT>(P, row, *T, d, cta);
            if (!alone)
                for (int i = lane; i < k; i += 32)
                    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(cluster_addr(&T->gathered[cta.rank * k + i], 0)),
                                 "l"(T->best[i])
                                 : "memory");
            __syncwarp();
        }
        if (!alone) {
            if (k) asm volatile("fence.acq_rel.cluster;" ::: "memory");
            __syncwarp();
            if (!exchange(P, S, cta, x++, p)) return false;
        }
    }
    const bool bad = row.state == kBad || (row.state == kLive && (p.n < 0 || p.m == -INFINITY));
    if (row.state == kLive && bad && lane == 0 && cta.rank == 0) atomicOr(P.status, SPECVERIFY_STATUS_BAD_LOGIT);
    const bool good = row.state == kLive && !bad;
    float lh = 0.0f, ll = 0.0f, lp = 0.0f, lo = 0.0f, H = 0.0f, lse = 0.0f;
    if (good) {
        ff_log(p.s, lh, ll);
        ff_logprob(P, row.zy, p.m, lh, ll, lp, lo);
        const float mean = p.t / p.s;
        H = lh - fmaf(mean, P.inv_hi, mean * P.inv_lo);
        float xh, xl;
        over_T(P, p.m, 0.0f, xh, xl);
        if (fabsf(xh) < INFINITY) ff_add(xh, xl, lh, ll, xh, xl);
        lse = xh;
    } else if (bad) {
        lp = H = lse = NAN;
    }
    if (lane == 0 && cta.rank == 0) {
        if (P.logprob) P.logprob[e] = lp;
        if (P.entropy) P.entropy[e] = H;
        if (!G && P.lse) P.lse[e] = lse;
        if (!G && P.rank) P.rank[e] = bad ? -1 : p.n;
    }
    if constexpr (!G) if (k && cta.rank == 0) {
        if (!good) {
            for (int i = lane; i < k; i += 32) {
                P.top_logprob[e * k + i] = bad ? NAN : -INFINITY;
                P.top_idx[e * k + i] = -1;
            }
        } else if (alone) {
            for (int i = lane; i < k; i += 32) write_top<DT>(P, e, i, T->best[i], p.m, lh, ll);
        } else {
            // each CTA's keys fall: a key's place is how many of each list are larger, found by halves
            for (int i = lane; i < k; i += 32) write_top<DT>(P, e, i, 0, p.m, lh, ll);
            __syncwarp();
            for (int i = lane; i < cta.cluster * k; i += 32) {
                const unsigned long long key = T->gathered[i];
                if (!key) continue;
                int place = i % k;
                for (int c = 0; c < cta.cluster && place < k; ++c) {
                    if (c == i / k) continue;
                    int lo_ = 0, hi_ = k;  // keys [0, lo_) are larger, [hi_, k) are not
                    while (lo_ < hi_) {
                        const int mid = (lo_ + hi_) >> 1;
                        if (T->gathered[c * k + mid] > key) lo_ = mid + 1;
                        else hi_ = mid;
                    }
                    place += lo_;
                }
                if (place < k) write_top<DT>(P, e, place, key, p.m, lh, ll);
            }
        }
    }
    if (G) {
        const float g = row.g, h = row.h;
        // p_v (-(g + h (ln p_v + H)) / T) with p_v = w / s and ln p_v = d / T - ln s
        const float inv_s = 1.0f / p.s;
        const float a = -(g + h * (H - lh)) * P.inv_hi * inv_s, b = -h * P.inv_hi * P.inv_hi * inv_s;
        if (lane == 0) {
            S.coef[d] = good ? make_float4(p.m, a, b, 0.0f) : make_float4(0.0f, NAN, NAN, 0.0f);
            mbar_arrive(smem_u32(&S.known[d]));
        }
        if (!wait_on(S.stored[d], parity, S.abort, P.status, P.wait_ns)) return false;
        const int y = row.y / Type<DT>::kPer;
        if (good && lane == 0 && y >= cta.slice0 && y < cta.slice0 + cta.slice_vecs) {
            const float py = ff_exp(lp, lo);
            const float s = py > 0.0f ? h * py * (lp + H) : 0.0f;
            store_logit<DT>(P.grad + e * P.grad_stride_bytes, row.y, (g * (1.0f - py) - s) * P.inv_hi);
        }
    }
    return true;
}

// The divergence over the list's tokens and the rest, see include/specverify.h. Logarithms are pairs of floats up to their
// differences: a small divergence is a difference of much larger terms.
template <int DT, bool G>
__device__ __forceinline__ bool finish_list(const TokenParams &P, Shared &S, SharedList &L, const Cta &cta, int d, uint32_t parity,
                                            Part p, int &x) {
    const Row &row = S.row[d];
    const long long e = row.entry;
    const int lane = cta.lane, K = P.K, kind = P.divergence;
    if (row.state == kLive && cta.cluster > 1 && !exchange(P, S, cta, x++, p)) return false;
    float zmax = -INFINITY;
    if (row.state == kLive)
        for (int j = lane; j < K; j += 32) zmax = fmaxf(zmax, L.z[d][j]);
    zmax = warp_max(zmax);
    const float M = fmaxf(p.m, zmax);
    const bool bad = row.state == kBad || (row.state == kLive && (p.n < 0 || M == -INFINITY));
    const bool good = row.state == kLive && !bad;
    if (row.state == kLive && bad && lane == 0 && cta.rank == 0) atomicOr(P.status, SPECVERIFY_STATUS_BAD_LOGIT);
    float loss = bad ? NAN : 0.0f, factor = 0.0f, C = 0.0f;
    const bool some = p.m > -INFINITY;  // the rest has mass
    if (good) {
        float Z = 0.0f;
        for (int j = lane; j < K; j += 32) Z += ex2_approx(fmaxf(L.z[d][j] - M, kFar) * P.c);
        Z = warp_sum(Z);
        if (some) Z = fmaf(p.s, ex2_approx(fmaxf(p.m - M, kFar) * P.c), Z);
        float zh, zl;
        ff_log(Z, zh, zl);
        float f = 0.0f, h = 0.0f, h_rest = 0.0f, q_rest = 0.0f;
        // outcome K is the rest
        for (int j = lane; j <= K; j += 32) {
            const bool rest = j == K;
            if (!rest && L.ids[d][j] < 0) continue;
            float qh, ql, lp = rest ? -INFINITY : L.lp[d][j];
            ff_logprob(P, rest ? p.m : L.z[d][j], M, zh, zl, qh, ql);
            if (rest && some) {
                float sh, sl;
                ff_log(p.s, sh, sl);
                if (qh > -INFINITY) ff_add(qh, ql, sh, sl, qh, ql);
            }
            const float q = ff_exp(qh, ql);
            float pr;
            if (rest) {
                pr = row.p_rest;
                lp = logf(kind == SPECVERIFY_RKL ? fmaxf(pr, 0x1p-20f) : pr);
            } else {
                pr = ff_exp(lp, 0.0f);
            }
            float fj = 0.0f, hj = 0.0f;
            if (kind == SPECVERIFY_FKL) {
                if (pr > 0.0f) fj = pr * ((lp - qh) - ql);
                hj = -pr;
            } else if (kind == SPECVERIFY_RKL) {
                if (q > 0.0f) fj = hj = q * ((qh - lp) + ql);
            } else if (kind == SPECVERIFY_TVD) {
                fj = 0.5f * fabsf(pr - q);
                hj = 0.5f * q * (q > pr ? 1.0f : q < pr ? -1.0f : 0.0f);
            } else {
                // ln(m / q) = ln(1 + b (p / q - 1)), and the other way round
                const float b = P.beta, r = (lp - qh) - ql;  // ln(p / q)
                if (q > 0.0f) hj = -(1.0f - b) * q * ln_mixed(b, pr > 0.0f ? r : -INFINITY);
                fj = hj;
                if (pr > 0.0f) fj -= b * pr * ln_mixed(1.0f - b, q > 0.0f ? -r : -INFINITY);
            }
            f += fj;
            h += hj;
            if (rest) {
                h_rest = hj;
                q_rest = q;
            } else {
                L.lp[d][j] = hj;  // what the gradient needs of it
                L.z[d][j] = q;
            }
        }
        loss = warp_sum(f);
        C = warp_sum(h);
        if (G) {
            h_rest = __shfl_sync(0xffffffffu, h_rest, K & 31);
            q_rest = __shfl_sync(0xffffffffu, q_rest, K & 31);
            factor = some ? row.g * P.inv_hi * (h_rest - q_rest * C) / p.s : 0.0f;
        }
    }
    if (lane == 0 && cta.rank == 0) P.loss[e] = loss;
    if (G) {
        if (lane == 0) {
            S.coef[d] = bad ? make_float4(0.0f, NAN, 0.0f, 0.0f) : make_float4(some ? p.m : 0.0f, factor, 0.0f, 0.0f);
            mbar_arrive(smem_u32(&S.known[d]));
        }
        if (!wait_on(S.stored[d], parity, S.abort, P.status, P.wait_ns)) return false;
        if (good)
            for (int j = lane; j < K; j += 32) {
                const int id = L.ids[d][j], v = id / Type<DT>::kPer;
                if (id >= 0 && v >= cta.slice0 && v < cta.slice0 + cta.slice_vecs)
                    store_logit<DT>(P.grad + e * P.grad_stride_bytes, id, row.g * P.inv_hi * (L.lp[d][j] - L.z[d][j] * C));
            }
    }
    return true;
}

template <int DT, bool LIST, bool G>
__device__ __forceinline__ void finish(const TokenParams &P, Shared &S, SharedTop *T, SharedList *L, const Cta &cta) {
    int r = 0, x = 0;
    for (long long e = cta.first; e < P.entries; e += cta.step, ++r) {
        const int d = cta.place(r);
        const uint32_t parity = cta.parity(r);
        if (!wait_on(S.row_full[d], parity, S.abort, P.status, P.wait_ns) ||
            !wait_on(S.summed[d], parity, S.abort, P.status, P.wait_ns))
            return;
        Part p{-INFINITY, 0.0f, 0.0f, 0};
        if (S.row[d].state == kLive) {
            if (cta.lane < kConsumers) p = S.part[d][cta.lane];
            p = warp_merge(p, P.c);
        }
        if (LIST ? !finish_list<DT, G>(P, S, *L, cta, d, parity, p, x) : !finish_token<DT, G>(P, S, T, cta, d, parity, p, x)) return;
        __syncwarp();
        if (cta.lane == 0) mbar_arrive(smem_u32(&S.row_free[d]));
    }
}

// ---------------------------------------------------------------------------

template <int DT, bool LIST, bool G>
__global__ void __launch_bounds__(kThreads, 2) token_kernel(const __grid_constant__ TokenParams P, const __grid_constant__ Plan plan) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *ring = smem;
    Shared &S = *reinterpret_cast<Shared *>(smem + (size_t)plan.slots * kChunkBytes);
    constexpr size_t kFixed = (sizeof(Shared) + 15) / 16 * 16;
    void *more = reinterpret_cast<uint8_t *>(&S) + kFixed;
    SharedTop *top = !LIST && !G && P.k > 0 ? static_cast<SharedTop *>(more) : nullptr;
    SharedList *list = LIST ? static_cast<SharedList *>(more) : nullptr;
    const int tid = threadIdx.x, warp = tid >> 5;

    Cta cta;
    cta.cluster = plan.cluster;
    cta.rank = plan.cluster > 1 ? (int)cluster_rank() : 0;
    cta.first = blockIdx.x / plan.cluster;
    cta.step = plan.clusters;
    const int vecs = (int)(((int64_t)P.V * Type<DT>::kSize + 15) / 16);
    cta.slice0 = min(vecs, cta.rank * plan.slice_vecs);
    cta.slice_vecs = min(vecs - cta.slice0, plan.slice_vecs);
    cta.chunks = (cta.slice_vecs + kChunkVecs - 1) / kChunkVecs;
    cta.lane = tid & 31;
    cta.depth_log = plan.depth_log;

    if (tid == 0) {
        for (int i = 0; i < plan.slots; ++i) {
            mbar_init(smem_u32(&S.full[i]), 1);
            mbar_init(smem_u32(&S.ready[i]), 1);
            mbar_init(smem_u32(&S.empty[i]), kConsumers);
        }
        for (int i = 0; i < kDepth; ++i) {
            mbar_init(smem_u32(&S.row_full[i]), 1);
            mbar_init(smem_u32(&S.row_free[i]), kConsumers + (LIST ? 3 : 2));
            mbar_init(smem_u32(&S.summed[i]), kConsumers);
            mbar_init(smem_u32(&S.known[i]), 1);
            mbar_init(smem_u32(&S.stored[i]), kConsumers);
            mbar_init(smem_u32(&S.bounded[i]), kConsumers);
        }
        mbar_init(smem_u32(&S.exchanged[0]), plan.cluster);
        mbar_init(smem_u32(&S.exchanged[1]), plan.cluster);
        S.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (LIST)
        for (int i = tid; i < kHash; i += kThreads) list->hash[i] = -1;
    __syncthreads();
    if (plan.cluster > 1) cluster_sync();
    after_previous();

    if (warp < kConsumers) consume<DT, LIST, G>(P, plan, S, top, ring, cta);
    else if (warp == kScout) scout<DT, LIST>(P, S, top, list, cta);
    else if (warp == kProducer) produce<DT>(P, plan, S, ring, cta);
    else if (LIST && warp == kPatcher) patch<DT>(P, plan, S, *list, ring, cta);
    else if (warp == kEpilogue) finish<DT, LIST, G>(P, S, top, list, cta);
    __syncwarp();
    // sums of other CTAs may still be on their way here where somebody gave up
    if (plan.cluster > 1) cluster_sync();
}

// ---------------------------------------------------------------------------
// host

size_t fixed_bytes(bool list, bool top) {
    return (sizeof(Shared) + 15) / 16 * 16 + (list ? sizeof(SharedList) : top ? sizeof(SharedTop) : 0);
}

constexpr int kHalfSmem = 113 * 1024, kFullSmem = 226 * 1024;  // of a CTA, two or one on an SM

// Rows over the GPU. The sums alone: one CTA a row where that fills the GPU, else as many as do (a power of two). With a
// gradient: the fewest that hold a row in their rings.
Plan make_plan(const TokenParams &P, int elem, bool list, bool grad, int num_sms) {
    const bool top = !list && !grad && P.k > 0;
    const int64_t vecs = ((int64_t)P.V * elem + 15) / 16;
    const int room = 2 * num_sms;
    Plan p{};
    p.depth_log = top ? 1 : 2;
    const int fixed = (int)fixed_bytes(list, top);
    const int half = (kHalfSmem - fixed) / kChunkBytes, full = std::min(kMaxSlots, (kFullSmem - fixed) / kChunkBytes);
    auto chunks = [&](int s) {
        const int64_t slice = ((vecs + s - 1) / s + 31) / 32 * 32;
        return (slice + kChunkVecs - 1) / kChunkVecs;
    };
    int S = 1;
    if (grad)
        while (S < kMaxCluster && 2 * chunks(S) > half) S *= 2;
    while (S < kMaxCluster && P.entries * S * 2 <= room && vecs >= 256 * S && (!top || P.k * S * 2 <= kGathered)) S *= 2;
    p.lag = grad && 2 * chunks(S) <= half;
    p.slots = !grad ? std::min(half, 8) : chunks(S) <= half ? half : full;
    p.cluster = S;
    p.slice_vecs = (int32_t)(((vecs + S - 1) / S + 31) / 32 * 32);
    const int resident = (p.slots > half ? num_sms : room) / S;
    p.clusters = (int32_t)std::min<int64_t>(P.entries, std::max(1, resident));
    p.smem = p.slots * kChunkBytes + fixed;
    return p;
}

template <int DT, bool LIST, bool G>
cudaError_t launch(const TokenParams &P, int num_sms, cudaStream_t s) {
    const Plan plan = make_plan(P, DT == SV_DT_FP32 ? 4 : 2, LIST, G, num_sms);
    return launch_after(token_kernel<DT, LIST, G>, dim3((unsigned)(plan.clusters * plan.cluster)), kThreads, plan.smem, s,
                        plan.cluster, P, plan);
}

template <int DT, bool LIST, bool G>
cudaError_t prepare() {
    cudaError_t e = cudaFuncSetAttribute(token_kernel<DT, LIST, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFullSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(token_kernel<DT, LIST, G>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

}  // namespace

cudaError_t prepare_token() {
    cudaError_t e = cudaSuccess;
    for (cudaError_t (*f)() : {prepare<SV_DT_FP32, false, false>, prepare<SV_DT_BF16, false, false>, prepare<SV_DT_FP32, false, true>,
                               prepare<SV_DT_BF16, false, true>, prepare<SV_DT_FP32, true, false>, prepare<SV_DT_BF16, true, false>,
                               prepare<SV_DT_FP32, true, true>, prepare<SV_DT_BF16, true, true>})
        if (e == cudaSuccess) e = f();
    return e;
}

cudaError_t launch_token_logprobs(const TokenParams &P, int dtype, int num_sms, cudaStream_t s) {
    return dtype == SV_DT_FP32 ? launch<SV_DT_FP32, false, false>(P, num_sms, s) : launch<SV_DT_BF16, false, false>(P, num_sms, s);
}

cudaError_t launch_token_logprobs_grad(const TokenParams &P, int dtype, int num_sms, cudaStream_t s) {
    return dtype == SV_DT_FP32 ? launch<SV_DT_FP32, false, true>(P, num_sms, s) : launch<SV_DT_BF16, false, true>(P, num_sms, s);
}

cudaError_t launch_distill(const TokenParams &P, int dtype, int num_sms, cudaStream_t s) {
    if (P.grad) return dtype == SV_DT_FP32 ? launch<SV_DT_FP32, true, true>(P, num_sms, s) : launch<SV_DT_BF16, true, true>(P, num_sms, s);
    return dtype == SV_DT_FP32 ? launch<SV_DT_FP32, true, false>(P, num_sms, s) : launch<SV_DT_BF16, true, false>(P, num_sms, s);
}

}  // namespace sv
