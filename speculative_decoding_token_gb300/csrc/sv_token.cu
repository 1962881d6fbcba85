// sv_token.cu -- log-probabilities of given tokens (with entropy, rank and top alternatives), their gradient, and the
// divergence of a draft's rows from the target's top tokens with its gradient. One CTA a row, several passes over it.
#include "sv_token.h"
#include "sv_stream.cuh"

namespace sv {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// The block's sum / maximum of x, in every thread (scratch: kWarps + 1 values).
template <class T, class F>
__device__ T block_fold(T x, T *scratch, F &&f) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x = f(x, __shfl_xor_sync(0xffffffffu, x, off));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    T r = scratch[0];
    for (int w = 1; w < kWarps; ++w) r = f(r, scratch[w]);
    return r;
}

template <int DT>
__device__ __forceinline__ void store_logit(char *row, int64_t v, float x) {
    if (DT == SV_DT_FP32) {
        reinterpret_cast<float *>(row)[v] = x;
    } else {
        uint16_t h;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
        reinterpret_cast<uint16_t *>(row)[v] = h;
    }
}

__device__ __forceinline__ unsigned long long order_key(float v, int i) {
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 orders as 0
    const uint32_t u = b & 0x80000000u ? ~b : b | 0x80000000u;
    return ((unsigned long long)u << 32) | (uint32_t)~i;
}

struct Shared {
    float f[kWarps];
    double d[kWarps];
    unsigned long long u[kWarps];
    int i[kWarps];
    int ids[kMaxList];
    float z[kMaxList];
};

// a logit's distance from the row's maximum, over T, in nats: to about 1e-7 of itself
__device__ __forceinline__ float scaled(const TokenParams &p, float d) {
    return d == -INFINITY ? d : fmaf(d, p.inv_hi, d * p.inv_lo);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(TokenParams p, int with_grad) {
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    auto add = [](auto a, auto b) { return a + b; };
    auto top = [](float a, float b) { return max_nan(a, b); };
    for (int64_t e = blockIdx.x; e < p.entries; e += gridDim.x) {
        const int y = p.tokens[e];
        int64_t row = e;
        if (p.row_off) row = p.row_off[e / p.M] + (p.path ? p.path[e] : e % p.M);
        bool bad = y != -1 && (y < 0 || y >= p.V || row < 0 || row >= p.rows);
        if (bad && tid == 0)
            atomicOr(p.status, y < 0 || y >= p.V ? SPECVERIFY_STATUS_BAD_TOKEN : SPECVERIFY_STATUS_BAD_ROW);
        const char *z = p.logits + row * p.stride_bytes;
        float m = 0.0f;
        if (!bad && y != -1) {
            m = -INFINITY;
            for (int v = tid; v < p.V; v += kThreads) m = max_nan(m, load_logit<DT>(z, v));
            m = block_fold(m, sh.f, top);
            bad = !(m > -INFINITY && m < INFINITY);
            if (bad && tid == 0) atomicOr(p.status, SPECVERIFY_STATUS_BAD_LOGIT);
        }
        if (bad || y == -1) {
            const float x = bad ? NAN : 0.0f;
            if (tid == 0) {
                if (p.logprob) p.logprob[e] = x;
                if (p.entropy) p.entropy[e] = x;
                if (p.lse) p.lse[e] = x;
                if (p.rank) p.rank[e] = bad ? -1 : 0;
            }
            for (int i = tid; i < p.k; i += kThreads) {
                p.top_logprob[e * p.k + i] = bad ? NAN : -INFINITY;
                p.top_idx[e * p.k + i] = -1;
            }
            if (with_grad)
                for (int v = tid; v < p.V; v += kThreads) store_logit<DT>(p.grad + e * p.grad_stride_bytes, v, x);
            continue;
        }
        const float zy = load_logit<DT>(z, y);
        float s = 0.0f, t = 0.0f;
        int before = 0;
        for (int v = tid; v < p.V; v += kThreads) {
            const float l = load_logit<DT>(z, v), d = fmaxf(l - m, -0x1p100f), w = ex2_approx(d * p.c);
            s += w;
            t = fmaf(w, d, t);
            before += l > zy || (l == zy && v < y);
        }
        s = block_fold(s, sh.f, add);
        t = block_fold(t, sh.f, add);
        const float ln_s = logf(s), H = ln_s - scaled(p, t / s), lp = scaled(p, zy - m) - ln_s;
        if (p.rank) before = block_fold(before, sh.i, add);
        if (tid == 0) {
            if (p.logprob) p.logprob[e] = lp;
            if (p.entropy) p.entropy[e] = H;
            if (p.lse) p.lse[e] = scaled(p, m) + ln_s;
            if (p.rank) p.rank[e] = before;
        }
        unsigned long long last = ~0ull;
        for (int i = 0; i < p.k; ++i) {
            unsigned long long best = 0;
            for (int v = tid; v < p.V; v += kThreads) {
                const unsigned long long key = order_key(load_logit<DT>(z, v), v);
                if (key < last && key > best) best = key;
            }
            last = best = block_fold(best, sh.u, [](unsigned long long a, unsigned long long b) { return a > b ? a : b; });
            if (tid == 0) {
                const int v = best ? (int)~(uint32_t)best : -1;
                p.top_idx[e * p.k + i] = v;
                p.top_logprob[e * p.k + i] = v < 0 ? -INFINITY : scaled(p, load_logit<DT>(z, v) - m) - ln_s;
            }
        }
        if (with_grad) {
            char *out = p.grad + e * p.grad_stride_bytes;
            const float g = p.g_logprob[e], h = p.g_entropy ? p.g_entropy[e] : 0.0f;
            const float inv_s = 1.0f / s;
            for (int v = tid; v < p.V; v += kThreads) {
                const float d = fmaxf(load_logit<DT>(z, v) - m, -0x1p100f), q = ex2_approx(d * p.c) * inv_s;
                float x = -q * g;
                if (v == y) x += g;
                if (h != 0.0f) x -= h * (q * (scaled(p, d) - ln_s + H));
                store_logit<DT>(out, v, x * p.inv_hi);
            }
        }
        __syncthreads();
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) distill_kernel(TokenParams p) {
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    auto add = [](auto a, auto b) { return a + b; };
    auto top = [](float a, float b) { return max_nan(a, b); };
    for (int64_t r = blockIdx.x; r < p.entries; r += gridDim.x) {
        const char *z = p.logits + r * p.stride_bytes;
        char *out = p.grad ? p.grad + r * p.grad_stride_bytes : nullptr;
        __syncthreads();
        int id = -1;
        float zk = -INFINITY, tk = -INFINITY;
        int bad = 0;
        if (tid < p.K) {
            id = p.ids[r * p.K + tid];
            sh.ids[tid] = id;
            if (id < -1 || id >= p.V) {
                bad = SPECVERIFY_STATUS_BAD_TOKEN;
            } else if (id >= 0) {
                zk = load_logit<DT>(z, id);
                tk = p.target_bf16 ? load_logit<SV_DT_BF16>(p.target, r * p.K + tid) : load_logit<SV_DT_FP32>(p.target, r * p.K + tid);
                if (!(zk < INFINITY) || !(tk < INFINITY)) bad = SPECVERIFY_STATUS_BAD_LOGIT;
            }
        }
        __syncthreads();
        if (id >= 0)
            for (int j = 0; j < tid; ++j)
                if (sh.ids[j] == id) bad = SPECVERIFY_STATUS_BAD_TOKEN;
        bad = block_fold(bad, sh.i, [](int a, int b) { return a | b; });
        const int live = block_fold(id >= 0 ? 1 : 0, sh.i, add);
        auto listed = [&](int v) {
            for (int j = 0; j < p.K; ++j)
                if (sh.ids[j] == v) return true;
            return false;
        };
        float m = -INFINITY, s = 0.0f;
        if (!bad && live) {
            for (int v = tid; v < p.V; v += kThreads)
                if (!listed(v)) m = max_nan(m, load_logit<DT>(z, v));
            m = block_fold(m, sh.f, top);
            if (!(m < INFINITY)) bad = SPECVERIFY_STATUS_BAD_LOGIT;
        }
        const float zmax = block_fold(id >= 0 ? zk : -INFINITY, sh.f, top);
        const float M = fmaxf(m, zmax);
        if (!bad && live && M == -INFINITY) bad = SPECVERIFY_STATUS_BAD_LOGIT;
        if (bad || !live) {
            if (bad && tid == 0) atomicOr(p.status, bad);
            if (tid == 0) p.loss[r] = bad ? NAN : 0.0f;
            if (out)
                for (int v = tid; v < p.V; v += kThreads) store_logit<DT>(out, v, bad ? NAN : 0.0f);
            continue;
        }
        if (m > -INFINITY)
            for (int v = tid; v < p.V; v += kThreads)
                if (!listed(v)) s += ex2_approx((load_logit<DT>(z, v) - m) * p.c);
        s = block_fold(s, sh.f, add);
        // K + 1 outcomes, in 64 bits: thread k < K has listed token k, thread K the rest
        const double inv = (double)p.inv_hi + (double)p.inv_lo;
        double x = -INFINITY;  // (z - M) / T
        if (id >= 0) x = ((double)zk - M) * inv;
        if (tid == p.K && s > 0.0f) x = ((double)m - M) * inv + log((double)s);
        const double lse = log(block_fold(x > -INFINITY ? exp(x) : 0.0, sh.d, add));
        const double lq = x - lse, q = lq > -INFINITY ? exp(lq) : 0.0;
        double lp = id >= 0 ? (double)tk : -INFINITY;
        if (p.form == SPECVERIFY_TARGET_LOGITS) {
            const float tm = block_fold((float)lp, sh.f, top);
            lp = tm > -INFINITY ? (lp - tm) * inv : lp;
            const double sum = block_fold(lp > -INFINITY ? exp(lp) : 0.0, sh.d, add);
            lp -= log(sum);
        }
        double pr = lp > -INFINITY ? exp(lp) : 0.0;
        const double sum = block_fold(pr, sh.d, add);
        if (tid == p.K) {
            pr = p.form == SPECVERIFY_TARGET_LOGITS ? 0.0 : fmax(1.0 - sum, 0.0);
            lp = log(p.divergence == SPECVERIFY_RKL ? fmax(pr, 0x1p-20) : pr);
        }
        double f = 0.0, h = 0.0;
        const bool mine = id >= 0 || tid == p.K;
        if (mine && p.divergence == SPECVERIFY_FKL) {
            if (pr > 0.0) f = pr * (lp - lq);
            h = -pr;
        } else if (mine && p.divergence == SPECVERIFY_RKL) {
            if (q > 0.0) f = h = q * (lq - lp);
        } else if (mine && p.divergence == SPECVERIFY_TVD) {
            f = 0.5 * fabs(pr - q);
            h = 0.5 * q * (q > pr ? 1.0 : q < pr ? -1.0 : 0.0);
        } else if (mine) {
            const double b = p.beta, lm = log(b * pr + (1.0 - b) * q);
            if (q > 0.0) h = (1.0 - b) * q * (lq - lm);
            f = h + (pr > 0.0 ? b * pr * (lp - lm) : 0.0);
        }
        const double loss = block_fold(f, sh.d, add), C = block_fold(h, sh.d, add);
        if (tid == 0) p.loss[r] = (float)loss;
        if (out) {
            const double w = (p.weight ? (double)p.weight[r] : 1.0) * inv, g = w * (h - q * C);
            __shared__ float scale;
            if (tid == p.K) scale = s > 0.0f ? (float)(g / s) : 0.0f;
            __syncthreads();
            const float a = scale;
            for (int v = tid; v < p.V; v += kThreads) {
                const float l = load_logit<DT>(z, v);
                if (!listed(v)) store_logit<DT>(out, v, m > -INFINITY ? a * ex2_approx((l - m) * p.c) : 0.0f);
            }
            __syncthreads();
            if (id >= 0) store_logit<DT>(out, id, (float)g);
        }
    }
}

int grid(int64_t entries, int num_sms) { return (int)(entries < 4 * num_sms ? entries : 4 * num_sms); }

}  // namespace

cudaError_t launch_token_logprobs(const TokenParams &p, int dtype, int num_sms, cudaStream_t s) {
    if (dtype == SV_DT_FP32) logprobs_kernel<SV_DT_FP32><<<grid(p.entries, num_sms), kThreads, 0, s>>>(p, 0);
    else logprobs_kernel<SV_DT_BF16><<<grid(p.entries, num_sms), kThreads, 0, s>>>(p, 0);
    return cudaGetLastError();
}

cudaError_t launch_token_logprobs_grad(const TokenParams &p, int dtype, int num_sms, cudaStream_t s) {
    if (dtype == SV_DT_FP32) logprobs_kernel<SV_DT_FP32><<<grid(p.entries, num_sms), kThreads, 0, s>>>(p, 1);
    else logprobs_kernel<SV_DT_BF16><<<grid(p.entries, num_sms), kThreads, 0, s>>>(p, 1);
    return cudaGetLastError();
}

cudaError_t launch_distill(const TokenParams &p, int dtype, int num_sms, cudaStream_t s) {
    if (dtype == SV_DT_FP32) distill_kernel<SV_DT_FP32><<<grid(p.entries, num_sms), kThreads, 0, s>>>(p);
    else distill_kernel<SV_DT_BF16><<<grid(p.entries, num_sms), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace sv
