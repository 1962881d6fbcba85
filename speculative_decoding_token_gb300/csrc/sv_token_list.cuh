// sv_token_list.cuh -- rows with lists (distillation): what the scout finds out of a
// list and what the epilogue makes of it, the divergence and its gradient.
#pragma once

#include "sv_token_state.cuh"

namespace sv {

namespace {

// What a row with a list is, the warp's work: its ids, where they are tokens.
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
            if (!(zk[i] < INFINITY) || !(t < (P.form == SPECVERIFY_TARGET_LOGITS ? INFINITY : 80.0f))) bits |= SPECVERIFY_STATUS_BAD_LOGIT;
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
    float lh = 0.0f, ll = 0.0f;
    zmax = warp_max(zmax);
    if (!bits) {
        if (P.form == SPECVERIFY_TARGET_LOGITS) {
            top = warp_max(top);
            float sum = 0.0f, suml = 0.0f;
            for (int j = lane; j < P.K; j += 32) {
                float h, l, wh, wl;
                if (llp[j] == -INFINITY) continue;
                ff_logprob(P, llp[j], top, 0.0f, 0.0f, h, l);
                ff_exp_pair(h, l, wh, wl);
                ff_add(sum, suml, wh, wl, sum, suml);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                ff_add(sum, suml, __shfl_xor_sync(all, sum, off), __shfl_xor_sync(all, suml, off), sum, suml);
            if (top == -INFINITY) bits = SPECVERIFY_STATUS_BAD_LOGIT;  // a target of nothing
            else ff_log_near(sum, suml, lh, ll);  // (the epilogue makes log-probabilities of them once more, in pairs)
            for (int j = lane; j < P.K; j += 32) {
                float h, l;
                ff_logprob(P, llp[j], top, lh, ll, h, l);
                lpr[j] = llp[j] == -INFINITY ? 0.0f : ff_exp(h, l);
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
        if (rkl) {
            row.p0_inv = 1.0f / p0;
            row.rest_inv = 1.0f / fmaxf(p_rest, 0x1p-20f);
        }
        row.tmax = top;
        row.t_h = lh;
        row.t_l = ll;
        row.zsum = zsum;
        row.zsum_l = zsum_l;
        row.cross = cross;
        if (bits) atomicOr(P.status, bits);
    }
}

// Puts the listed tokens' gradients in their places, once the consumers have stored the others'.
template <class Kd>
__device__ __forceinline__ void fix_list(const TokenParams &P, const Shared &S, const Lists &L, const Cta &cta, int d) {
    if (!S.good[d]) return;
    const float w = S.row[d].g * P.inv_hi;
    for (int j = cta.lane; j < P.K; j += 32) {
        const int at = d * L.stride + j, id = L.ids[at], v = id / Kd::kPer;
        if (id >= 0 && v >= cta.slice0 && v < cta.slice0 + cta.slice_vecs)
            store_logit<Kd::DT>(P.grad + S.row[d].entry * P.grad_stride_bytes, id, w * L.lp[at]);
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
    float Zh = 1.0f, Zl = 0.0f, oh = 0.0f, ol = 0.0f, t0 = 0.0f;
    if (good) {
        float dh, dl, wh = 0.0f, wl = 0.0f, mh, ml;
        ff_off_by(P, p.m, oh, ol);
        two_sum(lane & 1 ? p.m : row.zmax, -M, dh, dl);
        if (dh > P.far) {
            float xh, xl;
            over_T(P, dh, dl, xh, xl);
            if (lane & 1) ff_add(xh, xl, -oh, -ol, xh, xl);
            ff_exp_pair(xh, xl, wh, wl);
        }
        ff_mul(wh, wl, lane & 1 ? p.s : row.zsum, lane & 1 ? 0.0f : row.zsum_l, mh, ml);
        ff_add(mh, ml, __shfl_xor_sync(all, mh, 1), __shfl_xor_sync(all, ml, 1), Zh, Zl);
        if (Kd::Grad && early) {
            // Here sum h is known without a look at the list: -sum p, and sum q ln(q / p) by the scout's sums. The stores need
            // not wait for the divergence (2.5 us for a list of 128). q of that logit and of the rest, and ln(q / p):
            float qh, ql;
            {
                const float nh = lane & 1 ? mh : wh, nl = lane & 1 ? ml : wl, inv = 1.0f / Zh;
                qh = nh * inv;
                ql = (fmaf(-qh, Zh, nh) + fmaf(-qh, Zl, nl)) * inv;
            }
            if (kind == SPECVERIFY_FKL) {
                known(fmaf(qh, row.over, (qh - row.p_rest) + (ql - row.p_rest_l)));
            } else {
                const float ph = lane & 1 ? fmaxf(row.p_rest, 0x1p-20f) : row.p0;
                const float more = ((qh - ph) + (ql - (lane & 1 ? row.p_rest_l : row.p0_l))) * (lane & 1 ? row.rest_inv : row.p0_inv);
                const float t = fabsf(more) < 0.5f ? log1pf(more) : logf(qh) - (lane & 1 ? row.rest_h : row.lp0);
                // All relative to that logit's ln(q / p), t0, or gradients of a draft that is sure would be lost in it.
                const float q0 = __shfl_sync(all, qh, 0), qr = __shfl_sync(all, qh, 1), t1 = __shfl_sync(all, t, 1);
                t0 = __shfl_sync(all, t, 0);
                if (!(q0 > 0.0f)) t0 = 0.0f;
                const float gap = qr > 0.0f ? t1 - t0 : 0.0f, listed = q0 > 0.0f ? q0 * row.cross : 0.0f;
                C = fmaf(qr, gap, listed);
                known(qr > 0.0f ? qr * fmaf(gap, q0 * row.zsum, -listed) : 0.0f);
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
            if (qh > -INFINITY) {
                ff_add(sh, sl, -oh, -ol, sh, sl);
                ff_add(qh, ql, sh, sl, qh, ql);
            }
            q_rest = ff_exp(qh, ql);
        }
        r_rest = (row.rest_h - qh) + (row.rest_l - ql);
    }
    // h - q C where sum h = -sum p: q (1 + over) - p
    auto missing = [&](float pr, float q, float r) {
        return fmaf(q, row.over, fabsf(r) < 0.5f ? pr * expm1f(-r) : q - pr);
    };
    if (good) {
        float f = 0.0f, h = 0.0f, up = 0.0f, h_rest = 0.0f;
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
                float ph = L.lp[at], pl = 0.0f;
                if (P.form == SPECVERIFY_TARGET_LOGITS) ff_logprob(P, ph, row.tmax, row.t_h, row.t_l, ph, pl);
                r = (ph - h) + (pl - l);
            }
            float fj, hj;
            if (kind == SPECVERIFY_FKL) {
                fj = divergence_of(pr, q, r);
                hj = missing(pr, q, r);  // (with q C)
            } else if (kind == SPECVERIFY_RKL) {
                fj = divergence_of(q, rest ? fmaxf(pr, 0x1p-20f) : pr, -r);
                hj = q > 0.0f ? q * ((-r - t0) - C) : 0.0f;  // (with q C)
            } else if (kind == SPECVERIFY_TVD) {
                const bool near = fabsf(r) < 0.5f;
                fj = 0.5f * fabsf(near ? pr * expm1f(-r) : pr - q);
                hj = 0.5f * q * ((near ? r < 0.0f : q > pr) ? 1.0f : (near ? r > 0.0f : q < pr) ? -1.0f : 0.0f);
            } else {
                // ln(m / q) = ln(1 + b (p / q - 1)), and the other way round; each has a p, a q that is 0 or neither
                const float b = P.beta, m = b * pr + (1.0f - b) * q;
                const float u = q > 0.0f ? ln_mixed(b, pr > 0.0f ? r : -INFINITY) : 0.0f;
                const float v = pr > 0.0f ? ln_mixed(1.0f - b, q > 0.0f ? -r : -INFINITY) : 0.0f;
                hj = -(1.0f - b) * u;  // (less q C, and times q, below)
                fj = b * divergence_of(pr, m, -v) + (1.0f - b) * divergence_of(q, m, -u);
            }
            f += fj;
            if (kind == SPECVERIFY_TVD) {  // what C is less than a half (h > 0), and more than minus a half (h < 0)
                h += hj < 0.0f ? q : hj == 0.0f ? 0.5f * q : 0.0f;
                up += hj > 0.0f ? q : hj == 0.0f ? 0.5f * q : 0.0f;
            } else {
                h += hj;
            }
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
        if (Kd::Grad && !early) {
            C = warp_sum(h);
            h_rest = __shfl_sync(all, h_rest, K & 31);
            if (kind == SPECVERIFY_TVD) {
                up = warp_sum(up);
                auto left = [&](float hj, float q) { return hj > 0.0f ? q * C : hj < 0.0f ? -q * up : 0.5f * q * (C - up); };
                known(left(h_rest, q_rest));
                for (int j = lane; j < K; j += 32) L.lp[d * L.stride + j] = left(L.lp[d * L.stride + j], L.z[d * L.stride + j]);
            } else {
                // Relative to the likeliest outcome's, or gradients of a draft that is sure would be lost in it.
                float most = lane == 0 ? q_rest : 0.0f, ref = h_rest;
                for (int j = lane; j < K; j += 32) {
                    const int at = d * L.stride + j;
                    if (L.ids[at] >= 0 && L.z[at] > most) {
                        most = L.z[at];
                        ref = L.lp[at];
                    }
                }
                const unsigned who = __ballot_sync(all, most == warp_max(most));
                ref = __shfl_sync(all, ref, __ffs(who) - 1);
                C = lane == 0 ? q_rest * (h_rest - ref) : 0.0f;
                for (int j = lane; j < K; j += 32) {
                    const int at = d * L.stride + j;
                    if (L.ids[at] < 0) continue;
                    L.lp[at] -= ref;
                    C = fmaf(L.z[at], L.lp[at], C);
                }
                C = warp_sum(C);
                known(q_rest * ((h_rest - ref) - C));
                for (int j = lane; j < K; j += 32) L.lp[d * L.stride + j] = L.z[d * L.stride + j] * (L.lp[d * L.stride + j] - C);
            }
        }
    }
    if (lane == 0 && cta.rank == 0) P.loss[e] = loss;
    if (Kd::Grad && lane == 0) S.good[d] = good;
}

}  // namespace

}  // namespace sv
