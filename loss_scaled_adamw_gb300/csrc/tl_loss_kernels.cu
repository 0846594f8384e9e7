// tl_loss_kernels.cu - the objectives over vocabulary logits (include/tl_loss.h).
//
// Mathematics.  For one row x of V logits, it = 1 / temperature, M = max x:
//   S = sum_j exp((x_j - M) it),  lp = (x_y - M) it - log S,  q_j = exp((x_j - M) it) / S,
//   dL/dx_j = it g (1[j = y] - q_j),  g = dL/dlp.
// x - M is taken before the multiplication, so logits at the type's lowest value
// cannot overflow into a wrong finite result.
#include "tl_loss_internal.cuh"
#include "tl_internal.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tl {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// 2^v by the hardware unit (relative error about 2^-22).
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// A part of a row's sum: the largest element and the sum of exp((x - m) it) over
// the part.  A part without a finite element has m = -inf and s = 0 (s = NaN if it
// holds a NaN).
struct Part {
    float m, s;
};
__device__ __forceinline__ float part_ref(float m) { return m == kNegInf ? 0.0f : m; }
__device__ __forceinline__ Part join(Part a, Part b, float c2) {
    const float m = fmaxf(a.m, b.m), r = part_ref(m);
    return {m, __fmaf_rn(a.s, ex2((a.m - r) * c2), b.s * ex2((b.m - r) * c2))};
}
__device__ __forceinline__ Part warp_join(Part p, float c2) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        p = join(p, {__shfl_xor_sync(~0u, p.m, o), __shfl_xor_sync(~0u, p.s, o)}, c2);
    return p;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

__device__ __forceinline__ float teacher_logit(const LossArgs& a, int64_t at) {
    if (a.teacher_dtype == kBF16) return to_f(static_cast<const __nv_bfloat16*>(a.teacher)[at]);
    if (a.teacher_dtype == kF16) return to_f(static_cast<const __half*>(a.teacher)[at]);
    return static_cast<const float*>(a.teacher)[at];
}
__device__ __forceinline__ int64_t teacher_id(const LossArgs& a, int64_t at) {
    return a.id_bytes == 8 ? static_cast<const int64_t*>(a.tid)[at] : int64_t(static_cast<const int32_t*>(a.tid)[at]);
}

// The loss sums of one launch: each row group (a CTA or a cluster) adds its rows in
// order, writes a slot, and the group that takes the last ticket adds the slots.
struct LossSums {
    double loss = 0.0, first = 0.0, second = 0.0, count = 0.0;
};

__device__ __forceinline__ void write_result(const LossArgs& a, double loss, double first, double second,
                                             double count) {
    a.result[0] = float(loss / a.n);
    a.result[1] = float(first / a.n);
    a.result[2] = float(second / a.n);
    a.result[3] = float(count);
}

// Called by every thread of the group's first CTA.  Thread 0 holds the sums.
__device__ void pair_stage(const LossArgs& a, double* sh);

template <int OP>
__device__ void finish(const LossArgs& a, const LossSums& sum, int group, int ngroups) {
    __shared__ double sh[4 * 32];
    __shared__ bool last;
    const int tid = threadIdx.x, nw = blockDim.x >> 5, warp = tid >> 5, lane = tid & 31;
    __syncthreads();   // the CTA's row outputs come before its ticket
    if (tid == 0) {
        if (OP == kPolicy || OP == kDistill) {
            double* o = a.slots + 4 * int64_t(group);
            o[0] = sum.loss; o[1] = sum.first; o[2] = sum.second; o[3] = sum.count;
        }
        __threadfence();
        last = atomicAdd(a.ticket, 1u) == uint32_t(ngroups - 1);
        if (last) __threadfence();
    }
    __syncthreads();
    if (!last) return;
    if (OP == kPrefStat) {
        pair_stage(a, sh);
    } else {
        double v[4] = {0.0, 0.0, 0.0, 0.0};
        for (int i = tid; i < ngroups; i += blockDim.x)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] += __ldcg(a.slots + 4 * int64_t(i) + c);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[c] = warp_sum(v[c]);
            if (lane == 0) sh[c * 32 + warp] = v[c];
        }
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < nw; ++w)
                for (int c = 0; c < 4; ++c) v[c] += sh[c * 32 + w];
            write_result(a, v[0], v[1], v[2], v[3]);
        }
    }
    if (tid == 0) *a.ticket = 0;   // ready for the next call
}

// The pairs, by the last CTA of the first preference pass: a warp sums the
// log-ratios of one pair's two sequences (lanes strided, fp64), forms the pair's
// loss and its derivative, and writes the gradient factor of each of its rows.
__device__ void pair_stage(const LossArgs& a, double* sh) {
    const int tid = threadIdx.x, nw = blockDim.x >> 5, warp = tid >> 5, lane = tid & 31;
    const float step = (a.seed ? *a.seed : 1.0f) * a.inv_n * a.it;
    // rows outside every sequence keep w = 0, written by the row pass
    double loss = 0.0, margin = 0.0, won = 0.0, count = 0.0;
    for (int64_t p = warp; p < a.pairs; p += nw) {
        int64_t at[3];
        int64_t prev = 0;
        for (int i = 0; i < 3; ++i) {
            int64_t v = a.seq[2 * p + i];
            v = v < prev ? prev : v;
            at[i] = prev = v > a.rows ? a.rows : v;
        }
        double s[2];
        for (int i = 0; i < 2; ++i) {
            double v = 0.0;
            for (int64_t r = at[i] + lane; r < at[i + 1]; r += 32) v += double(__ldcg(&a.stat[r].ratio));
            s[i] = warp_sum(v);
        }
        const float h = float(double(a.beta) * (s[0] - s[1]));   // beta * h
        // log sg(h) = min(h, 0) - log1p(exp(-|h|)); sg(-h) and sg(h) without overflow
        const float t = expf(-fabsf(h)), l1 = log1pf(t);
        const float log_up = fminf(h, 0.0f) - l1, log_down = fminf(-h, 0.0f) - l1;
        const float big = 1.0f / (1.0f + t), small = t / (1.0f + t);
        const float down = h > 0.0f ? small : h <= 0.0f ? big : h, up = h > 0.0f ? big : h <= 0.0f ? small : h;
        const float l = -(1.0f - a.smooth) * log_up - (a.smooth > 0.0f ? a.smooth * log_down : 0.0f);
        const float dh = -a.beta * ((1.0f - a.smooth) * down - a.smooth * up);
        for (int i = 0; i < 2; ++i) {
            const float w = (i == 0 ? dh : -dh) * step;
            for (int64_t r = at[i] + lane; r < at[i + 1]; r += 32)
                if (a.target[r] >= 0) a.stat[r].w = w;
        }
        if (lane == 0) {
            if (a.loss) a.loss[p] = l;
            if (a.reward) {
                a.reward[2 * p] = float(double(a.beta) * s[0]);
                a.reward[2 * p + 1] = float(double(a.beta) * s[1]);
            }
            loss += l; margin += h; won += h > 0.0f ? 1.0 : 0.0; count += 1.0;
        }
    }
    if (lane == 0) { sh[warp] = loss; sh[32 + warp] = margin; sh[64 + warp] = won; sh[96 + warp] = count; }
    __syncthreads();
    if (tid == 0) {
        double v[4] = {0.0, 0.0, 0.0, 0.0};
        for (int c = 0; c < 4; ++c)
            for (int w = 0; w < nw; ++w) v[c] += sh[c * 32 + w];
        write_result(a, v[0], v[1], v[2], v[3]);
    }
}

// Policy: the row's loss and g = dL/dlp.
__device__ __forceinline__ float policy_row(const LossArgs& a, int64_t r, float lp, float& loss, float& surrogate,
                                            float& kl) {
    const float A = a.adv[r], ratio = expf(lp - a.old_logp[r]);
    const float freed = ratio * A, held = fminf(fmaxf(ratio, a.lo), a.hi) * A;
    // min(freed, held), a NaN of either kept
    surrogate = freed <= held ? -freed : freed > held ? -held : freed + held;
    float g = freed <= held ? -freed : freed > held ? 0.0f : freed + held;
    kl = 0.0f;
    if (a.ref_logp) {
        const float d = a.ref_logp[r] - lp, em = expm1f(d);
        kl = em - d;
        if (a.kl_weight > 0.0f) g = __fmaf_rn(a.kl_weight, -em, g);
    }
    loss = a.kl_weight > 0.0f ? __fmaf_rn(a.kl_weight, kl, surrogate) : surrogate;
    return g;
}

// The plain row kernel: one CTA per row at a time, elements strided over the
// threads, the row read once per use (maximum and sums, gradient).
template <typename T, int OP>
__global__ void __launch_bounds__(256) k_row_plain(const LossArgs a) {
    constexpr bool kTeach = OP == kDistill;
    __shared__ float sh_m[8], sh_s[8], sh_m1[8], sh_s1[8], sh_t[4][8];
    __shared__ int sh_id[kTeach ? kMaxTeacher + 1 : 1];
    __shared__ float sh_w[kTeach ? kMaxTeacher + 1 : 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float c2 = a.it * kLog2e;
    const float step = (a.dx && a.seed ? *a.seed : 1.0f) * a.inv_n;
    const bool kd_on = OP == kDistill && a.k > 0, ce_on = OP == kDistill && a.ce_weight > 0.0f;
    LossSums sum;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.ld;
        T* dx = a.dx ? static_cast<T*>(a.dx) + r * a.ldd : nullptr;
        const int64_t y = a.target ? a.target[r] : 0;
        __syncthreads();
        if (y < 0) {
            if (dx) for (int j = tid; j < a.vocab; j += 256) dx[j] = from_f<T>(0.0f);
            if (tid == 0) {
                if (OP != kDistill && a.logp) a.logp[r] = 0.0f;
                if ((OP == kPolicy || OP == kDistill) && a.loss) a.loss[r] = 0.0f;
                if (OP == kPrefStat) a.stat[r] = {0.0f, 0.0f, 0.0f, 0.0f};
            }
            continue;
        }
        float bad = y >= a.vocab ? __int_as_float(0x7fffffff) : 0.0f;   // NaN poisons the row
        const float xy = to_f(x[y < a.vocab ? y : 0]);
        Part p{kNegInf, 0.0f}, p1{kNegInf, 0.0f};
        for (int j = tid; j < a.vocab; j += 256) {
            const float v = to_f(x[j]);
            p = join(p, {v, v != v ? v : v == kNegInf ? 0.0f : 1.0f}, c2);
            if (ce_on) p1 = join(p1, {v, v != v ? v : v == kNegInf ? 0.0f : 1.0f}, kLog2e);
        }
        p = warp_join(p, c2);
        if (ce_on) p1 = warp_join(p1, kLog2e);
        // teacher: largest logit, sum of e, sum of e * (t - z)
        float tm = kNegInf, ts = 0.0f, td = 0.0f;
        if (kd_on) {
            float lm = kNegInf;
            for (int i = tid; i < a.k; i += 256) {
                const int64_t id = teacher_id(a, r * a.ldt + i);
                if (id >= a.vocab) bad = __int_as_float(0x7fffffff);
                const bool on = id >= 0 && id < a.vocab;
                sh_id[i] = on ? int(id) : -1;
                sh_w[i] = on ? teacher_logit(a, r * a.ldt + i) * a.it : kNegInf;
                if (on) lm = (sh_w[i] == sh_w[i]) ? fmaxf(lm, sh_w[i]) : sh_w[i];
            }
            for (int o = 16; o > 0; o >>= 1) {
                const float b = __shfl_xor_sync(~0u, lm, o);
                lm = lm != lm || b != b ? lm + b : fmaxf(lm, b);
            }
            if (lane == 0) sh_t[0][warp] = lm;
            bad = warp_sum(bad);
            if (lane == 0) sh_t[3][warp] = bad;
        }
        if (lane == 0) { sh_m[warp] = p.m; sh_s[warp] = p.s; sh_m1[warp] = p1.m; sh_s1[warp] = p1.s; }
        __syncthreads();
        p = warp_join({lane < 8 ? sh_m[lane] : kNegInf, lane < 8 ? sh_s[lane] : 0.0f}, c2);
        if (ce_on) p1 = warp_join({lane < 8 ? sh_m1[lane] : kNegInf, lane < 8 ? sh_s1[lane] : 0.0f}, kLog2e);
        if (kd_on) {
            for (int w = 0; w < 8; ++w) {
                const float b = sh_t[0][w];
                tm = tm != tm || b != b ? tm + b : fmaxf(tm, b);
                bad += sh_t[3][w];
            }
            for (int i = tid; i < a.k; i += 256) {
                const float t = sh_w[i];
                const float e = tm == kNegInf ? 0.0f : expf(t - tm);
                sh_w[i] = e;
                ts += e;
                if (e != 0.0f) td += e * (t - to_f(x[sh_id[i] < 0 ? 0 : sh_id[i]]) * a.it);
            }
            ts = warp_sum(ts);
            td = warp_sum(td);
            if (lane == 0) { sh_t[1][warp] = ts; sh_t[2][warp] = td; }
            __syncthreads();
            ts = td = 0.0f;
            for (int w = 0; w < 8; ++w) { ts += sh_t[1][w]; td += sh_t[2][w]; }
        }
        const float m = p.m == kNegInf ? __int_as_float(0x7fffffff) : p.m + bad;
        const float logs = logf(p.s), lp = (xy - m) * a.it - logs;
        if (OP == kLogprob || OP == kPrefStat) {
            if (tid == 0) {
                if (a.logp) a.logp[r] = lp;
                if (OP == kPrefStat) a.stat[r] = {m, 1.0f / p.s, 0.0f, a.ref_logp ? lp - a.ref_logp[r] : lp};
            }
        } else if (OP == kPolicy) {
            float loss, sur, kl;
            const float w = policy_row(a, r, lp, loss, sur, kl) * step * a.it;
            if (tid == 0) {
                if (a.logp) a.logp[r] = lp;
                if (a.loss) a.loss[r] = loss;
                sum.loss += loss; sum.first += sur; sum.second += kl; sum.count += 1.0;
            }
            if (dx) {
                const float kq = -w / p.s;
                for (int j = tid; j < a.vocab; j += 256) {
                    const float e = ex2((to_f(x[j]) - m) * c2);
                    dx[j] = from_f<T>(__fmaf_rn(e, kq, j == y ? w : 0.0f));
                }
            }
        } else {
            const bool row_kd = kd_on && ts != 0.0f;
            const float kd = row_kd ? (td / ts - tm - logf(ts) + m * a.it + logs) / (a.it * a.it) : 0.0f + bad;
            const float ce = ce_on ? logf(p1.s) - (xy - m) : 0.0f;
            const float loss = (row_kd ? a.kd_weight * kd : bad) + (ce_on ? a.ce_weight * ce : 0.0f);
            if (tid == 0) {
                if (a.loss) a.loss[r] = loss;
                sum.loss += loss; sum.first += kd; sum.second += ce; sum.count += 1.0;
            }
            if (dx) {
                const float wk = row_kd ? a.kd_weight * step / a.it : 0.0f, wc = ce_on ? a.ce_weight * step : 0.0f;
                const float kq = row_kd ? wk / p.s : 0.0f, cq = ce_on ? wc / p1.s : 0.0f;
                const int n = row_kd ? a.k : 0;
                __syncthreads();
                for (int i = tid; i < n; i += 256) sh_w[i] *= wk / ts;
                if (tid == 0 && ce_on) { sh_id[n] = bad == 0.0f ? int(y) : -1; sh_w[n] = wc; }
                const int entries = n + (ce_on ? 1 : 0);
                __syncthreads();
                // the listed entries' gradients first (their logits may be overwritten in place below)
                float fix[(kMaxTeacher + 256) / 256];
                unsigned mines = 0;
                int slot = 0;
                for (int i = tid; i < entries; i += 256, ++slot) {
                    float v = 0.0f;
                    const int id = sh_id[i];
                    bool mine = id >= 0;
                    for (int j = 0; j < entries && mine; ++j)
                        if (sh_id[j] == id) { if (j < i) mine = false; else v += sh_w[j]; }
                    if (mine) {
                        const float d = to_f(x[id]) - m;
                        v = (row_kd ? ex2(d * c2) * kq : 0.0f) + (ce_on ? ex2(d * kLog2e) * cq : 0.0f) - v;
                    }
                    fix[slot] = v;
                    mines |= unsigned(mine) << slot;
                }
                __syncthreads();
                for (int j = tid; j < a.vocab; j += 256) {
                    const float d = to_f(x[j]) - m;
                    dx[j] = from_f<T>((row_kd ? ex2(d * c2) * kq : bad) + (ce_on ? ex2(d * kLog2e) * cq : 0.0f));
                }
                __syncthreads();
                slot = 0;
                for (int i = tid; i < entries; i += 256, ++slot)
                    if (mines >> slot & 1) dx[sh_id[i]] = from_f<T>(fix[slot]);
            }
        }
    }
    if (OP != kLogprob) finish<OP>(a, sum, blockIdx.x, gridDim.x);
}

// Second preference pass: every element from its row's statistics.
template <typename T>
__global__ void __launch_bounds__(256) k_pref_grad_plain(const LossArgs a) {
    const float c2 = a.it * kLog2e;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.ld;
        T* dx = static_cast<T*>(a.dx) + r * a.ldd;
        const int64_t y = a.target[r];
        const RowStat st = a.stat[r];
        for (int j = threadIdx.x; j < a.vocab; j += 256) {
            float v = 0.0f;
            if (y >= 0 && st.w != 0.0f) v = __fmaf_rn(ex2((to_f(x[j]) - st.m) * c2), -st.w * st.rs, j == y ? st.w : 0.0f);
            dx[j] = from_f<T>(v);
        }
    }
}

template <typename T>
cudaError_t rows_by_op(int op, const LossArgs& a, int sm_count, cudaStream_t s) {
    const int64_t want = a.rows < 1 ? 1 : a.rows;
    const int grid = int(want < 4LL * sm_count ? want : 4LL * sm_count);
    switch (op) {
        case kLogprob: k_row_plain<T, kLogprob><<<grid, 256, 0, s>>>(a); break;
        case kPolicy: k_row_plain<T, kPolicy><<<grid, 256, 0, s>>>(a); break;
        case kPrefStat: k_row_plain<T, kPrefStat><<<grid, 256, 0, s>>>(a); break;
        default: k_row_plain<T, kDistill><<<grid, 256, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_loss_rows(int op, int dt, const LossArgs& a, int sm_count, cudaStream_t s) {
    if (dt == kF32) return rows_by_op<float>(op, a, sm_count, s);
    if (dt == kBF16) return rows_by_op<__nv_bfloat16>(op, a, sm_count, s);
    return rows_by_op<__half>(op, a, sm_count, s);
}

cudaError_t launch_pref_grad(int dt, const LossArgs& a, int sm_count, cudaStream_t s) {
    const int grid = int(a.rows < 8LL * sm_count ? a.rows : 8LL * sm_count);
    if (dt == kF32) k_pref_grad_plain<float><<<grid, 256, 0, s>>>(a);
    else if (dt == kBF16) k_pref_grad_plain<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
    else k_pref_grad_plain<__half><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace tl
