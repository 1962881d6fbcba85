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
    float bound;           // a number that k tokens reach
    uint32_t bound2, high2;
    float low, high;       // its class

    __device__ __forceinline__ Chooser(const TokenParams &P_, const Plan &plan, const char *row_, const SharedTop &T, int d, const Cta &cta_)
        : P(P_), row(row_), cta(cta_), log(plan.group_log) {
        set(from_order_bits(__reduce_min_sync(0xffffffffu, cta.lane < kConsumers ? T.bound[d][cta.lane] : ~0u)));
    }

    __device__ __forceinline__ void set(float x) {
        bound = x;
        const uint32_t upper = __float_as_uint(x) >> 16;
        bound2 = upper | upper << 16;
        low = high = __uint_as_float(upper << 16);
        if (DT == SV_DT_FP32 && fabsf(low) < INFINITY) {
            const float far = __uint_as_float(upper << 16 | 0xffffu);
            if (x < 0.0f) low = far;
            else high = far;
            if ((upper & 0x7fffu) == 0) {  // both zeros' classes are one
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

    __device__ __forceinline__ int rows() const { return (cta.chunks + (1 << log) - 1) >> log; }

    // A row of the groups' maxima, eight a lane: those above the class, or in it too.
    __device__ __forceinline__ uint32_t groups_of(const SharedTop &T, int d, int r, bool equal) const {
        const uint4 w = *reinterpret_cast<const uint4 *>(&T.most[d][r][cta.lane * 8]);
        return groups(w, false) | (equal ? groups(w, true) : 0u);
    }

    // A vector's tokens larger than the bound itself, or equal to it: bit u for token u. (What stands in for tokens that are
    // not there is -inf.)
    __device__ __forceinline__ uint32_t past_bound(const uint4 &w, int v, bool equal) const {
        float x[kPer];
        vec_floats<DT>(w, x);
        uint32_t in = 0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) in |= (equal ? x[u] == bound && v >= 0 && v * kPer + u < P.V : x[u] > bound) ? 1u << u : 0u;
        return in;
    }

    // Calls f(vectors, their indexes) over the vectors of all groups that may hold tokens larger than the bound.
    template <class F>
    __device__ __forceinline__ void each_past_bound(SharedTop &T, int d, F &&f) const {
        const bool equal = bound < high;
        for (int r = 0, n = rows(); r < n; ++r) {
            uint32_t in = groups_of(T, d, r, equal);
            int total, to = lanes_before(__popc(in), cta.lane, total);
            for (; in; in &= in - 1, ++to) T.kept[to] = (uint16_t)(r * kTeam + cta.lane * 8 + group_of(in));
            __syncwarp();
            each(total << (2 + log), [&](int j) { return vector(T.kept[j >> (2 + log)], j & ((4 << log) - 1)); }, f);
            __syncwarp();
        }
    }
};

// The k-th largest (k from 1) of the order bits that visit(f) calls f with, down to bit `last`, a digit of eight bits at a time
// by counting; false where there are fewer.
template <class Visit>
__device__ __forceinline__ bool nth_of(unsigned *bins, int k, int last, int lane, uint32_t &nth, Visit &&visit) {
    constexpr uint32_t all = 0xffffffffu;
    uint32_t mask = 0;
    nth = 0;
    for (int shift = 24; shift >= last; shift -= 8) {
        for (int i = lane; i < 256; i += 32) bins[i] = 0;
        __syncwarp();
        visit([&](uint32_t u) {
            if ((u & mask) == nth) atomicAdd(&bins[u >> shift & 255u], 1u);
        });
        __syncwarp();
        // lane l has digits 255 - 8 l and the seven below it
        int digit = 255 - 8 * lane, mine = 0, total;
#pragma unroll
        for (int q = 0; q < 8; ++q) mine += (int)bins[digit - q];
        int left = k - lanes_before(mine, lane, total);
        if (total < k) return false;
        const unsigned who = __ballot_sync(all, left > 0 && left <= mine);
        if (left > 0 && left <= mine)
            while (left > (int)bins[digit]) left -= (int)bins[digit--];
        k = __shfl_sync(all, left, __ffs(who) - 1);
        nth |= (uint32_t)__shfl_sync(all, digit, __ffs(who) - 1) << shift;
        mask |= 255u << shift;
        __syncwarp();
    }
    return true;
}

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

// The choice where the class is needed: `larger` keys above it are there, keys to T.keys[d], in any order, and how
// many; -1: too many groups, or tokens.
template <int DT>
__device__ __forceinline__ int choose_near(const TokenParams &P, const Plan &plan, const char *row, SharedTop &T, int d, const Cta &cta,
                                           int larger) {
    const Chooser<DT> choose(P, plan, row, T, d, cta);
    const int lane = cta.lane, k = P.k, log = plan.group_log, rows = choose.rows();
    // Groups above the class and, chunk after chunk, those in it until there are enough (of fp32: all).
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
    if (groups > kKept) return -1;
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
            choose.put(T.keys[d], w[q], v[q], in[q], to, kKeys);
            to += __popc(in[q]);
        }
        found += total;
        return found <= kKeys;
    });
    __syncwarp();
    return found <= kKeys ? found : -1;
}

// The choice where neither the groups above the bound's class nor those and the class's do: few tokens are left of the row, or
// left in few warps' vectors (the bound is -inf), or thousands are near it. Other warps wait for this one, and their waits have a
// limit: it raises the bound by the groups' maxima, and reads groups that reach it, not the row, six times at most (to count
// the order bits digit by digit where more than kKeys tokens are past the bound). Rows of 152064 logits, 256 at once, k = 20:
// fp32 with 4 tokens left 45 us (20.9 ms by the keys' bits over the whole row), 1024 neighbours 43, of bf16 50 (14 ms); fp32
// logits that are all the same 287 us, and 2.2 ms where all are in the bound's class and thousands past the bound. Unmasked: 37 and 31.
template <int DT>
__device__ __forceinline__ int choose_far(const TokenParams &P, const Plan &plan, const char *row, SharedTop &T, int d, const Cta &cta,
                                          unsigned found) {
    constexpr uint32_t all = 0xffffffffu;
    Chooser<DT> choose(P, plan, row, T, d, cta);
    using Kd = typename Chooser<DT>::Kd;
    const int lane = cta.lane, k = P.k, log = plan.group_log, rows = choose.rows();
    unsigned long long *keys = T.keys[d];
    unsigned *bins = reinterpret_cast<unsigned *>(T.best);  // (which is written later)
    static_assert(sizeof T.best >= 256 * sizeof *bins, "");
    uint32_t u;
    if (found >= (unsigned)k &&
        nth_of(bins, k, 16, lane, u, [&](auto &&f) {
            for (int r = 0; r < rows; ++r)
                for (uint32_t in = choose.groups_of(T, d, r, false); in; in &= in - 1)
                    f(order_bits(__uint_as_float((uint32_t)T.most[d][r][lane * 8 + choose.group_of(in)] << 16)));
        })) {
        // k groups reach a class above: its least number is a bound
        choose.set(from_order_bits(u >> 31 ? u : u | 0xffffu));
        choose.bound = choose.low;
    }
    auto collect = [&]() {  // the tokens larger than the bound, kKeys of them at most, and how many there are
        int n = 0;
        choose.each_past_bound(T, d, [&](const uint4 (&w)[4], const int (&v)[4]) {
            uint32_t in[4];
            int c = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                in[q] = choose.past_bound(w[q], v[q], false);
                c += __popc(in[q]);
            }
            int total, to = lanes_before(c, lane, total) + n;
            if (total == 0) return true;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                choose.put(keys, w[q], v[q], in[q], to, kKeys);
                to += __popc(in[q]);
            }
            n += total;
            return true;
        });
        __syncwarp();
        return n;
    };
    // (they are there already where none of the class are larger)
    int n = found < (unsigned)k && choose.bound == choose.high ? (int)found : collect();
    if (n > kKeys) {
        nth_of(bins, k, DT == SV_DT_FP32 ? 0 : 16, lane, u, [&](auto &&f) {
            choose.each_past_bound(T, d, [&](const uint4 (&w)[4], const int (&)[4]) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float x[Chooser<DT>::kPer];
                    vec_floats<DT>(w[q], x);
#pragma unroll
                    for (int i = 0; i < Chooser<DT>::kPer; ++i)
                        if (x[i] > choose.bound) f(order_bits(x[i]));
                }
                return true;
            });
        });
        choose.set(from_order_bits(DT == SV_DT_FP32 || u >> 31 ? u : u | 0xffffu));
        n = min(collect(), k);
    }
    // the first tokens that equal the bound, from the slice's start
    for (int r = 0; r < rows && n < k; ++r) {
        if (!__any_sync(all, choose.groups_of(T, d, r, true) != 0)) continue;
        const int first = (r << log) * Kd::kChunkVecs;
        choose.each(min(Kd::kChunkVecs << log, cta.slice_vecs - first), [&](int j) { return cta.slice0 + first + j; },
                    [&](const uint4 (&w)[4], const int (&v)[4]) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t in = choose.past_bound(w[q], v[q], true);
                int total;
                const int to = lanes_before(__popc(in), lane, total) + n;
                choose.put(keys, w[q], v[q], in, to, k);
                n = min(k, n + total);
            }
            return n < k;
        });
    }
    __syncwarp();
    return n;
}

// The rest of the choice where too few tokens are above the class, or too many. (One function: with a second call in it the
// epilogue's registers go to the stack, 26.2 us against 25.4 for 276 rows with 20 alternatives.)
template <int DT>
__device__ __noinline__ int choose_more(const TokenParams &P, const Plan &plan, const char *row, SharedTop &T, int d, const Cta cta,
                                        unsigned found) {
    int n = -1;
    if (found < (unsigned)P.k) n = choose_near<DT>(P, plan, row, T, d, cta, (int)found);
    if (n < 0) n = choose_far<DT>(P, plan, row, T, d, cta, found);
    return n;
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
