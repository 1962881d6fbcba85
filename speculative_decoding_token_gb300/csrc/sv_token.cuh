// sv_token.cuh -- the kernel of the calls on log-probabilities and distillation:
// log-probabilities of given tokens (with entropy, rank and top
// alternatives), the divergence of a draft's rows from its target's top tokens,
// and the gradients of both: one pass over rows of logits.
//
// A row is taken by a cluster of S CTAs, each a slice of it; S = 1 where there
// are rows enough. Slices come in chunks of 16 KiB by bulk copies into a ring of
// shared memory; a gradient's slice comes twice, the second time backwards and
// from L2. The warps of a CTA:
//   consumers (8)  a chunk's vectors, four a thread: a reference m near the
//                  maximum, the sums s of 2^x and t of 2^x x, x = z log2(e) / T
//                  relative to it; on the second reading, with the row's sums
//                  known, the gradient;
//   scout          the next row, and what its entry asks for (its token, or its
//                  list with the logits and probabilities of it);
//   producer       the copies;
//   patcher        (lists) takes the listed tokens out of a chunk that has
//                  arrived (-inf), so that the sums are over the rest alone;
//   top tokens     (the same warp, rows have one or the other) puts what the
//                  consumers have gathered in order;
//   epilogue       merges the warps' sums (and the cluster's), writes the results,
//                  and hands the consumers what a gradient's second reading needs.
// No warp waits for the end of a row but the consumers of a gradient. Rows are
// taken over from CTAs (clusters) that have not begun, one at a time, when the
// copies of the row before are on their way: CTAs differ by a sixth in speed.
//
// Bound by HBM: a row's logits once (twice and a gradient for gradients, one of
// the readings from L2). Measured, rows of 152064 bf16 logits: 2000 rows' log-
// probabilities and entropies 91 us (6.7 TB/s), with ranks 107, with 64 top
// tokens 125 (both by instructions); 2048 rows' gradients 198 (5.9 TB/s); 1111
// rows of 128256, divergences from lists of 64, 47.7 (5.4 TB/s).
#pragma once

#include "sv_token_list.cuh"
#include "sv_token_top.cuh"
#include "sv_tree.h"

#include <cuda_bf16.h>

#include <algorithm>

namespace sv {

namespace {

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

// A vector without its token e.
template <class Kd>
__device__ __forceinline__ uint4 without(const uint4 &w, int e) {
    auto word = [&](uint32_t x, int q) {
        if (Kd::DT == SV_DT_FP32) return q == e ? Kd::kNegInf : x;
        return q != e >> 1 ? x : e & 1 ? (x & 0xffffu) | 0xff800000u : (x & 0xffff0000u) | 0xff80u;
    };
    return make_uint4(word(w.x, 0), word(w.y, 1), word(w.z, 2), word(w.w, 3));
}

// The sums of a row's slice, chunk after chunk (a gradient's without the given token, which the epilogue adds: what the others
// have is 1 - p of it, also where that is 2^-40. 37 rows of 50257 with entropies 8.5 -> 8.8 us, 2048 of 152064 198.0 -> 198.4). A thread's reference m is its warp's maximum in the first chunk, and moves when
// a logit is 8 binades above it (TokenParams::lag): the sums are good whatever m is, and moving it for every new maximum costs
// 30 instructions in nearly every chunk (one of 32 lanes has a new maximum). What entropies lose by it is 8 2^-24.
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
    int own = -1;  // the chunk that has the given token, of the thread that does
    if (Kd::Grad && !Kd::List) {
        const int v = S.row[d].y / kPer - cta.slice0;
        if (v >= 0 && v % kTeam == tid) own = v / Kd::kChunkVecs;
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
        if (Kd::Grad && !Kd::List && i == own) {
            const int y = S.row[d].y, at = (y / kPer - cta.slice0) % Kd::kChunkVecs / kTeam;
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                if (j == at) w[j] = without<Kd>(w[j], y % kPer);
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
                    float f;
                    const float x = between(P, m, cm, f);
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
        if (Kd::Rank) {
            const int first = cta.slice0 + i * Kd::kChunkVecs;
            const bool inf = bound_before == bound_after;
            if (y_vec < first || (y_vec >= first + Kd::kChunkVecs && !inf)) {
                // One bound for the chunk, and nothing to count where no logit is larger. (2000 rows of 152064 bf16: 107 us for any
                // tokens, 104 for likely ones, 91 without ranks; 121 with a bound for each vector, and behind the exponentials.)
                const uint32_t bound = y_vec < first ? bound_after : bound_before;
                if (beyond<Kd::DT>(all, bound)) {
#pragma unroll
                    for (int j = 0; j < kVecs; ++j) above += count_above<Kd::DT>(w[j], bound);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    const int v = first + tid + j * kTeam;
                    if (v == y_vec || (inf && v < y_vec)) {
                        if (v < cta.slice0 + cta.slice_vecs) before += count_before<Kd>(w[j], S.row[d].zy, S.row[d].y, v * kPer);
                    } else {
                        above += count_above<Kd::DT>(w[j], v < y_vec ? bound_before : bound_after);
                    }
                }
            }
            if ((i & 1023) == 1023) {  // what is packed into half a word does not overflow
                before += counted<Kd::DT>(above);
                above = 0;
            }
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

// The gradient of a row's slice, 2^x (a + b x) with the sums' x, the last chunk first.
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
    if (near && Kd::List && !kFine) fa *= ex2_approx(m * P.c_lo);
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

template <class Kd>
__device__ __forceinline__ void scout(const TokenParams &P, const Plan &plan, Shared &S, const Lists &list, const Cta &cta,
                                      Entries &at) {
    Asked a;
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
        if (at.e < 0) return;
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
__device__ __forceinline__ void finish_token(const TokenParams &P, Shared &S, const Cta &cta, int d, Part p, const Part &own) {
    const Row &row = S.row[d];
    const long long e = row.entry;
    const int lane = cta.lane;
    float so = 0.0f, to = 0.0f;  // (a gradient's) sums of the others
    if (Kd::Grad) {
        const float m = fmaxf(p.m, own.m);
        float fo, fy;
        const float xo = between(P, p.m, m, fo), xy = between(P, own.m, m, fy);
        so = fo * p.s;
        to = fo * fmaf(xo, p.s, p.t);
        p = Part{m, fmaf(fy, own.s, so), fmaf(fy, fmaf(xy, own.s, own.t), to), min(p.n, own.n)};
    }
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
    float mh = lh, ml = ll;  // of the sum relative to p.m
    if (good) {
        float oh, ol;
        ff_off_by(P, p.m, oh, ol);
        ff_add(lh, ll, -oh, -ol, mh, ml);
        ff_logprob(P, row.zy, p.m, mh, ml, lp, lo);
    } else if (bad) {
        lp = H = NAN;
    }
    if (lane == 0 && cta.rank == 0) {
        if (P.logprob) P.logprob[e] = lp;
        if (P.entropy) P.entropy[e] = H;
        if (!Kd::Grad && P.lse) {
            float xh = 0.0f, xl = 0.0f;
            if (good) {
                over_T(P, p.m, 0.0f, xh, xl);
                if (fabsf(xh) < INFINITY) ff_add(xh, xl, mh, ml, xh, xl);
            }
            P.lse[e] = bad ? NAN : xh;
        }
        if (Kd::Rank) P.rank[e] = bad ? -1 : p.n;
    }
    if (Kd::Grad && lane == 0) {
        // g (1 - p) - h p (ln p + H), where 1 - p is the others' share and ln p + H that times (ln p - the mean of their ln p_v):
        // of a likely token the differences would leave little
        const float share = so * inv_s;
        float s = row.g;
        if (Kd::Ent) {
            const float ln = share < 0.5f ? log1pf(-share) : lp, mean = fmaf(__fdividef(to, so), kLn2Hi, -lh);
            if (share > 0.0f && lp > -INFINITY) s = fmaf(-row.h * ff_exp(lp, lo), ln - mean, s);
        }
        S.fix[d] = s * share * P.inv_hi;
        S.good[d] = good;
    }
}

// The top tokens of every row, beside the epilogue.
template <class Kd>
__device__ __forceinline__ void finish_top(const TokenParams &P, const Plan &plan, Shared &S, SharedTop &T, const Cta &cta) {
    const int lane = cta.lane, k = P.k;
    int live = 0;
    for (int r = 0;; ++r) {
        const int d = cta.place(r);
        if (!wait_bar(S.row_full[d], cta.parity(r), S, P)) return;
        const Row &row = S.row[d];
        const int state = row.state;
        if (state == kEnd) return;
        if (!wait_bar(S.summed[d], cta.parity(r), S, P)) return;
        if (state == kLive) {
            select_top<Kd::DT>(P, plan, row.z, T, d, cta);
            if (cta.cluster > 1) {
                for (int i = lane; i < k; i += 32)
                    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(cluster_addr(&T.gathered[cta.rank * k + i], 0)),
                                 "l"(T.best[i])
                                 : "memory");
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                __syncwarp();
                if (lane == 0) cluster_arrive(S.gathered, 0);
            }
        }
        if (cta.rank == 0) {
            Part p{-INFINITY, 0.0f, 0.0f, 0};
            if (state == kLive && cta.cluster > 1) {
                if (!wait_bar(S.gathered, 0, S, P)) return;  // a cluster of such rows has one
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                first_keys(T.gathered, cta.cluster * k, k, T.best, lane);
                if (!receive<Kd>(P, S, cta, live++, p)) return;
            } else if (state == kLive) {
                if (lane < kConsumers) p = S.part[d][lane];
                p = warp_fold<Kd>(P, p);
            }
            const bool good = state == kLive && p.n >= 0 && p.m > -INFINITY;
            float lh = 0.0f, ll = 0.0f;
            if (good) {
                float oh, ol;
                ff_off_by(P, p.m, oh, ol);
                ff_log(p.s, lh, ll);
                ff_add(lh, ll, -oh, -ol, lh, ll);
            }
            for (int i = lane; i < k; i += 32) {
                if (good) {
                    write_top<Kd::DT>(P, row.entry, i, T.best[i], p.m, lh, ll);
                } else {
                    P.top_logprob[row.entry * k + i] = state == kSkip ? -INFINITY : NAN;
                    P.top_idx[row.entry * k + i] = -1;
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&S.row_free[d]));
    }
}

// Puts the given token's gradient in its place, once the consumers have stored the others'.
template <class Kd>
__device__ __forceinline__ void fix_token(const TokenParams &P, const Shared &S, const Cta &cta, int d) {
    const int y = S.row[d].y, v = y / Kd::kPer;
    if (cta.lane == 0 && S.good[d] && v >= cta.slice0 && v < cta.slice0 + cta.slice_vecs)
        store_logit<Kd::DT>(P.grad + S.row[d].entry * P.grad_stride_bytes, y, S.fix[d]);
}

template <class Kd>
__device__ __forceinline__ void finish(const TokenParams &P, Shared &S, const Lists &L, const Cta &cta) {
    int live = 0;
    for (int r = 0;; ++r) {
        const int d = cta.place(r);
        const uint32_t parity = cta.parity(r);
        if (!wait_bar(S.row_full[d], parity, S, P)) return;
        const int state = S.row[d].state;
        if (state == kEnd) return;
        Part p{-INFINITY, 0.0f, 0.0f, 0};
        if (!wait_bar(S.scouted[d], parity, S, P)) return;
        Part own{-INFINITY, 0.0f, 0.0f, 0};  // (a gradient's) given token, as a sum relative to it
        if (Kd::Grad && !Kd::List && state == kLive) {
            const float z = S.row[d].zy;
            if (z < INFINITY) {
                const float x = plain(P, z) ? fmaf(z, P.c, -scaled(P, z)) : 0.0f, w = ex2_approx(x);
                if (z > -INFINITY) own = Part{z, w, w * x, 0};
            } else {
                own.n = -1;  // a bad one
            }
        }
        if (!wait_bar(S.summed[d], parity, S, P)) return;
        if (state == kLive && cta.cluster > 1) {
            if (!receive<Kd>(P, S, cta, live++, p)) return;
        } else if (state == kLive) {
            if (cta.lane < kConsumers) p = S.part[d][cta.lane];
            p = warp_fold<Kd>(P, p);
        }
        if (Kd::List) finish_list<Kd>(P, S, L, cta, d, p);
        else finish_token<Kd>(P, S, cta, d, p, own);
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
            mbar_init(smem_u32(&S.row_free[i]), kConsumers + (Kd::List || Kd::Top ? 3 : 2));
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
    else if (Kd::List && warp == kBeside) patch<Kd>(P, plan, S, list, smem, cta);
    else if (warp == kEpilogue) finish<Kd>(P, S, list, cta);
    else if constexpr (Kd::Top) finish_top<Kd>(P, plan, S, *top, cta);
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

// Rows over the GPU. One CTA a row where there are rows for every CTA that fits, else as many as do (a power of two). A
// gradient's rows go through L2 between their readings: no more of them at once than it holds well. room: the clusters of 2^i
// CTAs that fit at once.
template <class Kd>
Plan make_plan(const TokenParams &P, const int (&room)[5]) {
    const int64_t vecs = ((int64_t)P.V * Kd::kSize + 15) / 16;
    Plan p{};
    p.depth_log = Kd::Top ? 1 : 2;
    p.list_stride = Kd::List ? (P.K + 31) / 32 * 32 : 0;
    const int fixed = (int)((sizeof(Shared) + 15) / 16 * 16) +
                      (Kd::List ? kHashBytes + p.list_stride * kListBytes : Kd::Top ? (int)((sizeof(SharedTop) + 15) / 16 * 16) : 0);
    int log = 0;
    if (Kd::Grad)
        while (log < 4 && (int64_t)room[log] * vecs * 16 > kRereadBytes) ++log;
    const int64_t least = Kd::Top ? kLeastTop : 128;  // vectors of a slice
    while (log < 4 && P.entries <= room[log + 1] && vecs >> (log + 1) >= least && (!Kd::Top || P.k << (log + 1) <= kGathered)) ++log;
    p.cluster = 1 << log;
    p.slice_vecs = (int32_t)(((vecs + p.cluster - 1 >> log) + 31) / 32 * 32);
    const int words = log ? (2 * kConsumers * Kd::kWords * 8) << log : 0;
    static_assert(!Kd::Top || sizeof(Shared) + 15 + sizeof(SharedTop) + 15 + 2 * kConsumers * Kd::kWords * 8 * kMaxCluster +
                                      4 * Kd::kChunkBytes <= kHalfSmem, "kGroupRows");
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

// A kernel's set-up on the current device, at a handle's first call that takes it. Not at the handle's making (18 kernels of five
// questions each: a program's first handle took 3.8 ms instead of 2.4, also where it only verifies), and not once for a process:
// another device has other room.
template <class Kd>
cudaError_t prepare(TokenRoom &room) {
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
        int fit = 0;
        e = cudaOccupancyMaxActiveClusters(&fit, token_kernel<Kd>, &cfg);
        room.clusters[log].store(fit, std::memory_order_relaxed);
    }
    if (e == cudaSuccess) room.known.store(true, std::memory_order_release);
    return e;
}

template <class Kd>
cudaError_t launch(const TokenParams &P, TokenRooms &rooms, cudaStream_t s) {
    TokenRoom &room = rooms.of[Kd::kId];
    if (!room.known.load(std::memory_order_acquire)) {
        const cudaError_t e = prepare<Kd>(room);
        if (e != cudaSuccess) return e;
    }
    int clusters[5];
    for (int log = 0; log < 5; ++log) clusters[log] = room.clusters[log].load(std::memory_order_relaxed);
    const Plan plan = make_plan<Kd>(P, clusters);
    return launch_after(token_kernel<Kd>, dim3((unsigned)(plan.clusters * plan.cluster)), kThreads, plan.smem, s, plan.cluster, P,
                        plan);
}

}  // namespace

}  // namespace sv
