// sv_token_top.cuh -- the top tokens of a row, chosen from the maxima of groups of
// its vectors that the sums leave behind (sv_token.cuh).
#pragma once

#include "sv_token_state.cuh"

#include <cuda_bf16.h>

namespace sv {

namespace {

// Puts those of n keys that are among the first k in their places in `best`: a key's place is how many are larger, counted by
// 32 N keys' lanes at a time over all n, two at a load. (64 keys take N = 2 some 250 cycles of independent instructions. A bitonic
// network has 21 steps of two shuffles that wait on one another: 2.3 us for k = 20,
// here 1.5; 6.7 us for k = 64, 5.9 beside other work.)
template <int N>
__device__ __forceinline__ void place_keys(const unsigned long long *keys, int n, int k, unsigned long long *best, int lane) {
    int there = 0;
    for (int b = 0; b < n; b += 32 * N) {
        unsigned long long x[N];
        int before[N];
#pragma unroll
        for (int q = 0; q < N; ++q) {
            x[q] = b + 32 * q + lane < n ? keys[b + 32 * q + lane] : 0;
            before[q] = 0;
        }
#pragma unroll 4
        for (int i = 0; i < n; i += 2) {
            const ulonglong2 o = *reinterpret_cast<const ulonglong2 *>(keys + i);
            const unsigned long long second = i + 1 < n ? o.y : 0;
#pragma unroll
            for (int q = 0; q < N; ++q) before[q] += (o.x > x[q] ? 1 : 0) + (second > x[q] ? 1 : 0);
        }
#pragma unroll
        for (int q = 0; q < N; ++q) {
            if (x[q] && before[q] < k) best[before[q]] = x[q];
            there += __popc(__ballot_sync(0xffffffffu, x[q] != 0));
        }
    }
    for (int i = there + lane; i < k; i += 32) best[i] = 0;
    __syncwarp();
}

// The first k of n keys, all of them different (but 0, which is none), in order; 0 where there are no more.
__device__ __noinline__ void first_keys(const unsigned long long *keys, int n, int k, unsigned long long *best, int lane) {
    if (n <= 32) place_keys<1>(keys, n, k, best, lane);
    else if (n <= 64) place_keys<2>(keys, n, k, best, lane);
    else place_keys<4>(keys, n, k, best, lane);
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
                if (to < kKept) T.kept[to] = (uint16_t)(r * kTeam + lane * 8 + choose.group_of(in));
            groups += total;
        }
        __syncwarp();
        bool ok = groups <= kKept;
        if (ok)
            choose.each(groups << (2 + log), [&](int j) { return choose.vector(T.kept[j >> (2 + log)], j & ((4 << log) - 1)); },
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

// The k best keys of the CTA's slice, in order, to T.best (0 where there are none).
template <int DT>
__device__ __forceinline__ void select_top(const TokenParams &P, const Plan &plan, const char *row, SharedTop &T, int d, const Cta &cta) {
    const unsigned found = *(volatile unsigned *)&T.found[d];
    int n = (int)found;
    if (found < (unsigned)P.k || found > (unsigned)kKeys) n = choose_more<DT>(P, plan, row, T, d, cta, found);
    __syncwarp();
    first_keys(T.keys[d], n, P.k, T.best, cta.lane);
    if (cta.lane == 0) T.found[d] = 0;  // for the row after the next
}

}  // namespace

}  // namespace sv
