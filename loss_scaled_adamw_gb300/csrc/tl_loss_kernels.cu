// tl_loss_kernels.cu - the objectives over vocabulary logits (include/tl_loss.h).
//
// Mathematics.  For one row x of V logits, it = 1 / temperature, M = max x:
//   S = sum_j exp((x_j - M) it),  lp = (x_y - M) it - log S,  q_j = exp((x_j - M) it) / S,
//   dL/dx_j = it g (1[j = y] - q_j),  g = dL/dlp.
#include "tl_loss_internal.cuh"
#include "tl_internal.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tl {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
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

// Exponents.  With c2 = it log2(e) an element's exponential is taken as 2^(x c2 - u), u the
// whole number next to m c2 of the largest element m (or one near it): one multiply-add, and sums over parts
// with other u join by exact powers of two.  From |m c2| = 2^24 on (u would not be exact;
// logits at a type's lowest value, masks of -1e9) it is 2^((x - m) c2) instead.  (At
// temperature 1, for the cross-entropy, the exponent is x log2(e).)
__device__ __forceinline__ bool big(float m, float c2) { return !(fabsf(m) * fmaxf(c2, kLog2e) < 16777216.0f); }
__device__ __forceinline__ float anchor(float m, float c2) { return rintf(m * c2); }

// 2^n for a whole n <= 0.
__device__ __forceinline__ float power_of_two(float n) { return __int_as_float((int(fmaxf(n, -127.0f)) + 127) << 23); }

// A part of a row (a thread's or a warp's elements) has its largest element m and its sum s
// of exponentials.  A part without an element above -inf takes 0 in the place of m, so its s
// is 0 (NaN if it holds a NaN), and parts join without -inf - -inf.
__device__ __forceinline__ float part_ref(float m) { return m == kNegInf ? 0.0f : m; }
// The exponential of x in a part whose largest element is m.
__device__ __forceinline__ float power(float x, float m, float c2) {
    return ex2(big(m, c2) ? (x - m) * c2 : __fmaf_rn(x, c2, -anchor(m, c2)));
}
// What brings a part's sum from its largest element m to the joined one.
__device__ __forceinline__ float rescale(float m, float to, float c2) {
    if (m == kNegInf) return 1.0f;   // an empty part's 0 (or NaN) stays
    if (!big(to, c2) && !big(m, c2)) return power_of_two(anchor(m, c2) - anchor(to, c2));
    if (!big(to, c2)) return ex2(__fmaf_rn(m, c2, -anchor(to, c2)));   // from 2^((x - m) c2)
    // to 2^((x - to) c2)
    return ex2((m - to) * c2 - (big(m, c2) ? 0.0f : __fmaf_rn(m, c2, -anchor(m, c2))));
}

// log2 of s exponentials' sum as a whole part and the rest, so that neither is rounded to the
// size of the whole.
__device__ __forceinline__ void log2_parts(float s, float& n, float& rest) {
    const int e = (__float_as_int(s) >> 23) - 127;
    const bool usual = s > 1e-30f && s < 1e30f;
    n = usual ? float(e) : 0.0f;
    rest = log2f(usual ? __int_as_float(__float_as_int(s) - (e << 23)) : s);
}
// a + b, and what its rounding left out.
__device__ __forceinline__ float sum_parts(float a, float b, float& left) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    left = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
    return s;
}
// log(exponential of x / s) in a part whose largest element is m, with anchor u; c: the scale
// of x times log2(e).
__device__ __forceinline__ float log_share(float x, float m, float u, float c, bool far, float s) {
    float n, rest;
    log2_parts(s, n, rest);
    const float plain = ((far ? (x - m) * c - n : __fmaf_rn(x, c, -(u + n))) - rest) * kLn2;
    // The same with the error of each step carried along, so that the log-probability is rounded
    // once at its own size: of the 3.7e-7 rms that three roundings left on 128,256 entries a
    // long sequence's reward is a sum.
    constexpr double kExactLn2 = 0.693147180559945309;
    constexpr float kLn2Low = float(kExactLn2 - double(kLn2));
    const float z = far ? x - m : x, b = far ? n : u + n;
    const float p = __fmul_rn(z, c), pe = __fmaf_rn(z, c, -p);
    float de, he;
    const float d = sum_parts(p, -b, de), h = sum_parts(d, -rest, he);
    const float low = __fadd_rn(__fadd_rn(pe, de), he);
    const float r = __fmul_rn(h, kLn2), re = __fmaf_rn(h, kLn2, -r);
    const float lp = __fadd_rn(r, __fadd_rn(re, __fmaf_rn(low, kLn2, __fmul_rn(h, kLn2Low))));
    return fabsf(lp) < INFINITY ? lp : plain;   // infinities leave no error to carry
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

// Some of a row's teacher entries (a thread's, a warp's, all): their largest logit m, the sum s
// of their exponentials, the student's logit z at the first of them, and d, the sum of the
// exponentials times (t - m) - (x - z).  The divergence is made of d and of two logarithms of
// shares (log_share): differences of logits only, so that an offset common to a row is not
// rounded into its loss.  (z is of the first entry, not of m's: it is known before the maximum.)
// An entry that the student excludes (x of -inf) has z = 0 and d = inf.
// Without entries m is -inf and s 0; a NaN s makes the row NaN.
struct __align__(16) TeacherPart {
    float m, s, d, z;
};
__device__ __forceinline__ TeacherPart teacher_entry(float t, float e, float x) {
    const bool out = x == kNegInf;
    return {t, e, out && e != 0.0f ? INFINITY : 0.0f, out ? 0.0f : x};
}
// p.d against another reference (m, z), times f.
__device__ __forceinline__ float moved(const TeacherPart& p, float f, float m, float z) {
    return f != 0.0f && p.s != 0.0f ? f * __fmaf_rn(p.s, (p.m - m) - (p.z - z), p.d) : 0.0f;
}

__device__ __forceinline__ float teacher_logit(const LossArgs& a, int64_t at) {
    if (a.teacher_dtype == kBF16) return to_f(static_cast<const __nv_bfloat16*>(a.teacher)[at]);
    if (a.teacher_dtype == kF16) return to_f(static_cast<const __half*>(a.teacher)[at]);
    return static_cast<const float*>(a.teacher)[at];
}
__device__ __forceinline__ int64_t teacher_id(const LossArgs& a, int64_t at) {
    return a.id_bytes == 8 ? static_cast<const int64_t*>(a.tid)[at] : int64_t(static_cast<const int32_t*>(a.tid)[at]);
}

// Named barriers: `count` threads take part; arrive does not wait.
__device__ __forceinline__ void bar_sync(int id, int count) {
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int count) {
    __syncwarp();
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// The loss sums of one launch: each row group adds its rows in order and writes a slot, and
// the group that takes the last ticket adds the slots.
struct LossSums {
    double loss = 0.0, first = 0.0, second = 0.0, count = 0.0;
};

// Whether this group is the last of the launch to come here (lane 0 of one warp asks).
__device__ __forceinline__ bool last_group(const LossArgs& a, int ngroups) {
    __threadfence();
    if (atomicAdd(a.ticket, 1u) != uint32_t(ngroups - 1)) return false;
    __threadfence();
    *a.ticket = 0;   // ready for the next call
    return true;
}

// By the statistics warp of a group's first CTA, whose first lane holds the sums: the element
// warps may still be writing gradients.
__device__ __forceinline__ void finish_sums(const LossArgs& a, const LossSums& sum, int group, int ngroups) {
    const int lane = threadIdx.x & 31;
    double2* const slots = reinterpret_cast<double2*>(a.slots);
    bool last = false;
    if (lane == 0) {
        slots[2 * group] = make_double2(sum.loss, sum.first);
        slots[2 * group + 1] = make_double2(sum.second, sum.count);
        last = last_group(a, ngroups);
    }
    if (!__shfl_sync(~0u, last, 0)) return;
    __syncwarp();   // the first lane's acquire holds for all: a shuffle orders no memory
    double v[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
    for (int i = lane; i < ngroups; i += 32) {
        const double2 p = __ldcg(slots + 2 * i), q = __ldcg(slots + 2 * i + 1);
        v[0] += p.x; v[1] += p.y; v[2] += q.x; v[3] += q.y;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = warp_sum(v[c]);
    const double mine = lane == 0 ? v[0] : lane == 1 ? v[1] : lane == 2 ? v[2] : v[3];
    if (lane < 4) a.result[lane] = float(lane < 3 ? mine * a.per_n : mine);
}

// The four sums over the first B threads of the CTA, and the result.
template <int B> __device__ __forceinline__ void write_sums(const LossArgs& a, double (&v)[4]) {
    constexpr int nw = B / 32;
    __shared__ double sh[4 * nw];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        v[c] = warp_sum(v[c]);
        if (lane == 0) sh[4 * warp + c] = v[c];
    }
    bar_sync(5, B);
    if (warp == 0) {   // lane 4 w + c: sum c of warp w (at most 8 warps)
        double s = lane < 4 * nw ? sh[lane] : 0.0;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(~0u, s, o);
        if (lane < 4) a.result[lane] = float(lane < 3 ? s * a.per_n : s);
    }
}

template <int B> __device__ void pair_stage(const LossArgs& a);

// The preference's first pass: called by every thread of a group's first CTA; the rows'
// statistics are written.  Thread TAKER takes the group's ticket.
template <int B, int TAKER> __device__ void finish_pairs(const LossArgs& a, int ngroups) {
    __shared__ bool last;
    __syncthreads();
    if (threadIdx.x == TAKER) last = last_group(a, ngroups);
    __syncthreads();
    if (last && threadIdx.x < B) pair_stage<B>(a);
}

// The pairs, by the last CTA of the first preference pass: a warp sums the log-ratios of
// one pair's two sequences (lanes strided, eight loads under way, fp64), forms the pair's loss
// and its derivative, and writes the gradient factor of each of its rows.
template <int B> __device__ void pair_stage(const LossArgs& a) {
    constexpr int nw = B / 32, U = 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float step = (a.seed ? *a.seed : 1.0f) * a.inv_n * a.it;
    // rows outside every sequence keep w = 0, written by the row pass
    double loss = 0.0, margin = 0.0, won = 0.0, count = 0.0;
    for (int64_t p = warp; p < a.pairs; p += nw) {
        int64_t at[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) at[i] = a.seq[2 * p + i];
        int64_t prev = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            at[i] = at[i] < prev ? prev : at[i];
            at[i] = prev = at[i] > a.rows ? a.rows : at[i];
        }
        double s[2] = {0.0, 0.0};
        for (int64_t r = at[0] + lane; r < at[2]; r += 32 * U) {
            float q[U];
#pragma unroll
            for (int j = 0; j < U; ++j) q[j] = r + 32 * j < at[2] ? __ldcg(&a.stat[r + 32 * j].ratio) : 0.0f;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (r + 32 * j < at[1]) s[0] += double(q[j]); else s[1] += double(q[j]);
            }
        }
        s[0] = warp_sum(s[0]);
        s[1] = warp_sum(s[1]);
        const float h = float(double(a.beta) * (s[0] - s[1]));   // beta * h
        // log sg(h) = min(h, 0) - log1p(exp(-|h|)); sg(-h) and sg(h) without overflow
        const float t = expf(-fabsf(h)), l1 = log1pf(t);
        const float log_up = fminf(h, 0.0f) - l1, log_down = fminf(-h, 0.0f) - l1;
        const float big = 1.0f / (1.0f + t), small = t / (1.0f + t);
        const float down = h > 0.0f ? small : h <= 0.0f ? big : h, up = h > 0.0f ? big : h <= 0.0f ? small : h;
        const float l = -(1.0f - a.smooth) * log_up - (a.smooth > 0.0f ? a.smooth * log_down : 0.0f);
        const float w = -a.beta * ((1.0f - a.smooth) * down - a.smooth * up) * step;
        // all rows of the pair; those that are ignored are zeros whatever their factor
        for (int64_t r = at[0] + lane; r < at[2]; r += 32) a.stat[r].w = r < at[1] ? w : -w;
        if (lane == 0) {
            if (a.loss) a.loss[p] = l;
            if (a.reward) {
                a.reward[2 * p] = float(double(a.beta) * s[0]);
                a.reward[2 * p + 1] = float(double(a.beta) * s[1]);
            }
            loss += l; margin += h; won += h > 0.0f ? 1.0 : 0.0; count += 1.0;
        }
    }
    double v[4] = {loss, margin, won, count};   // the first lanes' pairs
    write_sums<B>(a, v);
}

// Policy: the row's loss and g = dL/dlp.
__device__ __forceinline__ float policy_row(const LossArgs& a, float lp, float old, float adv, float ref, float& loss,
                                            float& surrogate, float& kl) {
    const float ratio = expf(lp - old);
    const float freed = ratio * adv, held = fminf(fmaxf(ratio, a.lo), a.hi) * adv;
    // min(freed, held), a NaN of either kept
    surrogate = freed <= held ? -freed : freed > held ? -held : freed + held;
    float g = freed <= held ? -freed : freed > held ? 0.0f : freed + held;
    kl = 0.0f;
    if (a.ref_logp) {
        const float d = ref - lp, em = expm1f(d);
        kl = em - d;
        if (a.kl_weight > 0.0f) g = __fmaf_rn(a.kl_weight, -em, g);
    }
    loss = a.kl_weight > 0.0f ? __fmaf_rn(a.kl_weight, kl, surrogate) : surrogate;
    return g;
}

// ---------------------------------------------------------------------------
// 16-byte vectors of logits
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint4 ld16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st16(void* p, uint4 v) {
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kEmpty = 0xff800000u;   // -inf
    static __device__ __forceinline__ float top(uint4 v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ void wide(uint4 v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 narrow(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static constexpr uint32_t kEmpty = 0xff80ff80u;
    static __device__ __forceinline__ __nv_bfloat162 b2(uint32_t v) { return *reinterpret_cast<__nv_bfloat162*>(&v); }
    static __device__ __forceinline__ float top(uint4 v) {
        const __nv_bfloat162 m = __hmax2(__hmax2(b2(v.x), b2(v.y)), __hmax2(b2(v.z), b2(v.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ void one(uint32_t v, float& lo, float& hi) {
        lo = __uint_as_float(v << 16);
        hi = __uint_as_float(v & 0xffff0000u);
    }
    static __device__ __forceinline__ void wide(uint4 v, float (&f)[8]) {
        one(v.x, f[0], f[1]); one(v.y, f[2], f[3]); one(v.z, f[4], f[5]); one(v.w, f[6], f[7]);
    }
    static __device__ __forceinline__ uint32_t back(float lo, float hi) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
        return make_uint4(back(f[0], f[1]), back(f[2], f[3]), back(f[4], f[5]), back(f[6], f[7]));
    }
};
template <> struct Vec<__half> {
    static constexpr int N = 8;
    static constexpr uint32_t kEmpty = 0xfc00fc00u;
    static __device__ __forceinline__ __half2 h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
    static __device__ __forceinline__ float top(uint4 v) {
        const __half2 m = __hmax2(__hmax2(h2(v.x), h2(v.y)), __hmax2(h2(v.z), h2(v.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ void one(uint32_t v, float& lo, float& hi) {
        const float2 w = __half22float2(h2(v));
        lo = w.x;
        hi = w.y;
    }
    static __device__ __forceinline__ void wide(uint4 v, float (&f)[8]) {
        one(v.x, f[0], f[1]); one(v.y, f[2], f[3]); one(v.z, f[4], f[5]); one(v.w, f[6], f[7]);
    }
    static __device__ __forceinline__ uint32_t back(float lo, float hi) {
        const __half2 r = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
        return make_uint4(back(f[0], f[1]), back(f[2], f[3]), back(f[4], f[5]), back(f[6], f[7]));
    }
};

// Where a row's elements lie: `head` elements up to the first 16-byte boundary, `body`
// whole vectors from there, and a tail.  The head and tail elements ("edges", fewer than
// 2 N) are held one per thread by the first CTA of the group; [lo, hi) are the vectors of
// this CTA's share.  The share begins `off` places behind a 128-byte boundary; those places
// are empty, so that a warp's copies and stores cover whole lines.
template <typename T> struct Place {
    int head, body, edges, lo, hi, off;
    __device__ __forceinline__ Place(const T* row, int vocab, int rank, int clog) {
        constexpr int N = Vec<T>::N;
        const int ph = int((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % N);
        head = ph == 0 ? 0 : min(N - ph, vocab);
        body = (vocab - head) / N;
        edges = vocab - body * N;
        const int share = (body + (1 << clog) - 1) >> clog;
        lo = min(body, rank * share);
        hi = min(body, lo + share);
        off = int(reinterpret_cast<uintptr_t>(row + head + lo * N) >> 4) & 7;
    }
    __device__ __forceinline__ int edge_at(int i) const { return i < head ? i : i + body * Vec<T>::N; }
    // whether element j is this CTA's: edge element `i`, or in vector `i` of the row
    __device__ __forceinline__ bool owns(int j, int rank, bool& at_edge, int& i) const {
        i = (j - head) / Vec<T>::N;
        at_edge = j < head || i >= body;
        if (at_edge) i = j < head ? j : j - body * Vec<T>::N;
        return at_edge ? rank == 0 : i >= lo && i < hi;
    }
};

// Vector stores need the gradient row at the logits' phase; other rows are stored by elements.
template <typename T>
__device__ __forceinline__ void store_vec(T* dst, uint4 v, bool whole) {
    if (whole) {
        st16(dst, v);
    } else {
        T e[Vec<T>::N];
        *reinterpret_cast<uint4*>(e) = v;
#pragma unroll
        for (int i = 0; i < Vec<T>::N; ++i) dst[i] = e[i];
    }
}
template <typename T>
__device__ __forceinline__ bool same_phase(const T* x, const T* dx) {
    return ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(dx)) & 15u) == 0;
}

// ---------------------------------------------------------------------------
// The row kernel
// ---------------------------------------------------------------------------

constexpr int kMaxClusterLog = 3, kMaxCluster = 1 << kMaxClusterLog;

__device__ __forceinline__ uint32_t cluster_rank() { uint32_t r; asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r)); return r; }
// The cluster's barrier in halves.  Only the statistics warps write into other CTAs, so
// only their arrival releases: a releasing arrival of the others would wait for the
// gradient's stores.
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive_relaxed() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(const void* smem, uint32_t rank, float4 v) {
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(smem)), to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// The lanes' teacher parts joined.
__device__ __forceinline__ TeacherPart warp_join(const TeacherPart& p, float c2) {
    TeacherPart r;
    const unsigned has = __ballot_sync(~0u, p.m > kNegInf && p.d < INFINITY);
    r.z = __shfl_sync(~0u, p.z, has ? __ffs(has) - 1 : 0);
    r.m = warp_max(p.m);
    const float f = rescale(p.m, part_ref(r.m), c2);
    r.s = warp_sum(p.s * f);
    r.d = warp_sum(moved(p, f, r.m, r.z));
    return r;
}

// The sum at temperature 1 beside the one at tau (distillation with both terms).  For tau
// = 2 or 4 (POW) its exponentials are powers of the tempered ones; else (POW = 0) they are
// taken from the logits.
template <int POW> __device__ __forceinline__ float untempered(float e, float x, float v) {
    if (POW == 0) return ex2(__fmaf_rn(x, kLog2e, -v));
    const float r = e * e;
    return POW == 4 ? r * r : r;
}
// A vector's exponentials added up, before they meet a running sum.  One at a time onto it, the
// small ones of a long row fall below half of its last place more often than they round up: a
// spread of 5 bits over 128,256 entries cost the sum 1.5e-7 in the mean (0.7 in place of 1 as
// the temperature of logits with a deviation of 2.5).  Four vectors at a time leave nothing
// of that, and it is the same number of additions.
template <int N> __device__ __forceinline__ float tree_sum(const float (&e)[N]) {
    const float a = (e[0] + e[1]) + (e[2] + e[3]);
    if constexpr (N == 8) return a + ((e[4] + e[5]) + (e[6] + e[7]));
    return a;
}
// The same of the untempered ones; powers fold into multiply-adds.
template <int POW, int N> __device__ __forceinline__ float untempered_sum(const float (&e)[N], const float (&x)[N], float v) {
    if constexpr (POW == 0) {
        float w[N];
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = untempered<POW>(e[j], x[j], v);
        return tree_sum(w);
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float r = POW == 4 ? e[j] * e[j] : e[j];
        sum = j == 0 ? r * r : __fmaf_rn(r, r, sum);
    }
    return sum;
}
// e kq plus the untempered exponential times cq.
template <int POW> __device__ __forceinline__ float mix(float e, float x, float v, float kq, float cq) {
    if (POW == 2) return e * __fmaf_rn(e, cq, kq);
    return __fmaf_rn(untempered<POW>(e, x, v), cq, e * kq);
}
// The exponent's reference at temperature 1 for a largest element m, u = anchor(m, c2).
template <int POW> __device__ __forceinline__ float untempered_ref(float m, float u) {
    return POW == 0 ? anchor(m, kLog2e) : u * float(POW);
}
template <int POW> __device__ __forceinline__ float rescale1(float m, float to, float c2) {
    if (m == kNegInf) return 1.0f;
    const float ref = untempered_ref<POW>(m, anchor(m, c2));
    if (!big(to, c2)) {
        const float end = untempered_ref<POW>(to, anchor(to, c2));
        return big(m, c2) ? ex2(__fmaf_rn(m, kLog2e, -end)) : power_of_two(ref - end);
    }
    return ex2((m - to) * kLog2e - (big(m, c2) ? 0.0f : __fmaf_rn(m, kLog2e, -ref)));
}
// The same two exponentials of one element where m may be big.
template <int POW> __device__ __forceinline__ float power1(float e, float x, float m, float c2) {
    return big(m, c2) ? ex2((x - m) * kLog2e) : untempered<POW>(e, x, untempered_ref<POW>(m, anchor(m, c2)));
}

__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

constexpr int kMaxRingBytes = 220 * 1024;   // dynamic shared memory: tiles and teacher entries

// A tile is kTileVecs vectors per thread, kStages of them are in shared memory.
constexpr int kTileVecs = 8, kStages = 3;
constexpr int kSingle = -1;   // POW of the kernels with one sum per row
constexpr int64_t kRowsInL2 = 48 << 20;

// How a launch lays its rows out: threads per CTA, and CTAs per row (2^clog).
struct RowShape {
    int threads, clog;
};

// A group of 2^clog CTAs takes one row at a time, each CTA a contiguous share of the row's
// vectors.  The share comes through shared memory in tiles, copied asynchronously ahead of
// their use; a thread copies the vectors that it will itself use, so a tile needs no
// barrier.
//
// B threads work on the elements, in two passes over a row: A keeps each thread's running
// maximum and sum, B writes the gradient.  One more warp has the statistics: it joins the
// warps' parts, exchanges the CTAs' parts through distributed shared memory, and works
// out the row's loss and gradient factors (by all warps they cost as many instructions as
// the elements).
//
// A share of at most one tile stays in shared memory between its passes (kept): the row is
// read once, and its pass B comes after pass A of the next row, so that the element warps
// do not wait for the factors.  Longer shares are streamed a second time, out of L2 (see
// shape_for), and their pass B comes at once: with two rows under way per group the second
// read misses L2 (2,432 rows of 50,000: 63 % of the copy rate, one at a time 79 %).
//
// What bounds it: the longest rows, memory (4,096 x 128,256 bf16, one in eight ignored:
// log-probabilities 135 us, 6.8 TB/s; policy 322 us, 6.1 TB/s, 92 % of the copy rate);
// rows below about 10,000 entries, the chain from a row's last element to its factors, with
// 16 instructions per element in the passes.  Ring and grid: three tiles of 32 KB per CTA of
// 256 threads, two CTAs per SM, measured against 4 and 16 vectors per thread, two and four
// tiles, three CTAs per SM, 64 to 512 threads, and groups of 1 to 8 CTAs.
// POW: distillation with both terms at temperatures that differ, two sums per row (DUAL).  4,096 x
// 128,256 bf16, 64 entries: 398 us at temperature 2 (POW 2), 418 at 4 (POW 4), 451 at 3 (POW 0, a
// second exponential per element), 377 at 1 (one sum).  The 16-bit
// POW 0 forms spill 4 to 28 bytes per thread, that of POW 4 with 128 threads 8 to 12.
template <typename T, int OP, int B, int POW>
__global__ void __launch_bounds__(B + 32, B == 256 ? 2 : B == 128 ? 4 : 6) k_row(const LossArgs a, const int clog) {
    constexpr int N = Vec<T>::N, U = 4, tile = B * kTileVecs, ST = kStages, nw = B / 32;
    constexpr bool DUAL = POW != kSingle;
    constexpr bool kTeach = OP == kDistill;
    constexpr bool kGrad = OP == kPolicy || OP == kDistill;
    __shared__ float4 wparts[2][nw];                // by row parity, per warp: m, s, s at temperature 1
    __shared__ TeacherPart tparts[2][kTeach ? nw : 1];
    __shared__ float4 cparts[2][kMaxCluster];       // per CTA of the group
    // Of four rows in turn: while a row is in pass A its predecessor is in pass B and the one
    // before that has its listed elements written, and a warp may be a row ahead of another.
    __shared__ float4 fac[4][2];                    // gradient factors
    // [ST][tile] vectors; then [4][3][kpad] of id, t, x.  A copy of a warp into memory off a
    // 128-byte boundary takes twice the requests (4,096 x 128,256 bf16 policy: 361 us, on it 326).
    extern __shared__ __align__(128) uint4 ring[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = 1 << clog, rank = cluster > 1 ? int(cluster_rank()) : 0;
    const int group = int(blockIdx.x) >> clog, ngroups = int(gridDim.x) >> clog;
    float* const teach = reinterpret_cast<float*>(ring + ST * tile);
    const int kpad = (a.k + 3) & ~3;
    const float c2 = a.it * kLog2e;
    const bool kd_on = kTeach && a.k > 0, ce_on = kTeach && a.ce_weight > 0.0f;
    const bool grad = kGrad && a.dx != nullptr;
    const float kNaN = __int_as_float(0x7fffffff);
    LossSums sum;
    int par = 0, buf4 = 0;   // of the row: which of two, which of four
    int64_t ynext = a.target && group < a.rows ? a.target[group] : 0;
    // The dense gradient of one logit x: its exponentials times their factors.
    auto dense_value = [&](float x, float Mb, float kq, float cq) {
        const float e = power(x, Mb, c2);
        return DUAL ? __fmaf_rn(power1<POW>(e, x, Mb, c2), cq, e * kq) : e * kq;
    };
    // The label of row r, that of the group's next one under way.
    auto label = [&](int64_t r) {
        const int64_t y = ynext;
        if (a.target && r + ngroups < a.rows) ynext = a.target[r + ngroups];
        return y;
    };

    if (OP == kPrefStat) asm volatile("griddepcontrol.launch_dependents;");   // the gradient's kernel, see there

    if (warp == nw) {
        // ------------------------------------------------------------ the statistics warp
        const float step = (kGrad && a.seed ? *a.seed : 1.0f) * a.inv_n;
        const bool out = rank == 0 && lane == 0;
        if (cluster > 1) {   // every CTA of the group runs before any writes into another
            cluster_arrive();
            cluster_wait();
        }
        for (int64_t r = group; r < a.rows; r += ngroups) {
            const int64_t y = label(r);
            if (y < 0) {
                if (out) {
                    if (OP != kDistill && a.logp) a.logp[r] = 0.0f;
                    if (kGrad && a.loss) a.loss[r] = 0.0f;
                    if (OP == kPrefStat) a.stat[r] = {0.0f, 0.0f, 0.0f, 0.0f};
                }
                continue;
            }
            float xy = to_f(static_cast<const T*>(a.x)[r * a.ld + (y < a.vocab ? y : 0)]);
            float old = 0.0f, adv = 0.0f, refl = 0.0f;
            if (OP == kPolicy) {
                old = a.old_logp[r];
                adv = a.adv[r];
            }
            if (OP == kPolicy || OP == kPrefStat) refl = a.ref_logp ? a.ref_logp[r] : 0.0f;
            // x_y has arrived before this CTA lets any other overwrite the row in place
            xy = __shfl_sync(~0u, xy, 0);
            float S = 0.0f, S1 = 0.0f, M = kNegInf;
            auto join = [&](float4 p) {   // lane i holds part i, the others an empty one
                M = warp_max(p.x);
                S = warp_sum(p.y * rescale(p.x, part_ref(M), c2));
                if (DUAL) S1 = warp_sum(p.z * rescale1<POW>(p.x, part_ref(M), c2));
            };
            const float4 none = make_float4(kNegInf, 0.0f, 0.0f, 0.0f);
            bar_sync(1 + par, B + 32);
            join(lane < nw ? wparts[par][lane] : none);
            TeacherPart te{kNegInf, 0.0f, 0.0f, 0.0f};
            auto teacher = [&]() {
                if (lane < nw && lane * 32 < a.k) te = tparts[par][lane];
                te = warp_join(te, c2);
            };
            if (cluster > 1) {
                if (lane < cluster) store_remote(&cparts[par][rank], uint32_t(lane), make_float4(M, S, S1, 0.0f));
                cluster_arrive();
                if (kd_on) teacher();
                cluster_wait();
                join(lane < cluster ? cparts[par][lane] : none);
            } else if (kd_on) {
                teacher();
            }
            float bad = y >= a.vocab || M == kNegInf ? kNaN : 0.0f;
            const bool far = big(M, c2);
            const float u = anchor(M, c2);
            const float lp = log_share(xy, M, u, c2, far, S) + bad;
            if (OP == kLogprob || OP == kPrefStat) {
                bar_arrive(3 + par, B + 32);   // nothing for pass B
                if (out && a.logp) a.logp[r] = lp;
                if (OP == kPrefStat && out) a.stat[r] = {M + bad, 1.0f / S, 0.0f, lp - refl};
            } else if (OP == kPolicy) {
                float loss, sur, kl;
                const float w = policy_row(a, lp, old, adv, refl, loss, sur, kl) * step * a.it;
                // the label's element: w (1 - q)
                const float kq = -w / S;
                if (lane == 0) fac[buf4][0] = make_float4(M + bad, kq, 0.0f, __fmaf_rn(power(xy, M, c2), kq, w));
                bar_arrive(3 + par, B + 32);
                if (out) {
                    if (a.logp) a.logp[r] = lp;
                    if (a.loss) a.loss[r] = loss;
                    sum.loss += loss; sum.first += sur; sum.second += kl; sum.count += 1.0;
                }
            } else {
                // without a softmax of the student (a NaN or +inf logit) or the teacher: a row with neither
                // entries nor a cross-entropy takes nothing else from S
                if (!(S < INFINITY) || te.s != te.s) bad = kNaN;
                const bool row_kd = te.s != 0.0f;
                // factors of the exponentials at the temperature and at 1, and of the teacher's
                // (e_i = exp((t_i - te.m) it) times wp; 0: none)
                const float wk = row_kd ? a.kd_weight * step / a.it : 0.0f, wc = ce_on ? a.ce_weight * step : 0.0f;
                const float kq = wk / S + (DUAL ? 0.0f : wc / S) + bad;
                const float kq0 = row_kd || (!DUAL && ce_on) || bad != 0.0f ? kq : 0.0f, cq = DUAL ? wc / S1 : 0.0f;
                const float wp = row_kd ? wk / te.s : 0.0f;
                // the label's element: the teacher may list it too
                float at_label = 0.0f;
                if (ce_on && grad) {
                    const float* const tb = teach + buf4 * 3 * kpad;
                    for (int i = lane; i < (wp != 0.0f ? a.k : 0); i += 32)
                        if (__float_as_int(tb[i]) == int(y)) at_label = __fmaf_rn(wp, power(tb[kpad + i], part_ref(te.m), c2), at_label);
                    at_label = dense_value(xy, M + bad, kq0, cq) - (warp_sum(at_label) + wc);
                }
                if (lane == 0) {
                    fac[buf4][0] = make_float4(M + bad, kq0, cq, at_label);
                    fac[buf4][1] = make_float4(wp, te.m, anchor(te.m, c2), 0.0f);
                }
                bar_arrive(3 + par, B + 32);
                // kd = tau^2 (sum p ((t - te.m) - (x - te.z)) / tau + log p at te.m - log q at te.z)
                const float tau = 1.0f / a.it;
                const float logs = log_share(te.m, te.m, anchor(te.m, c2), c2, big(te.m, c2), te.s) - log_share(te.z, M, u, c2, far, S);
                const float kd = !row_kd ? bad : te.d == INFINITY ? te.d + bad : (te.d / te.s + logs * tau) * tau + bad;
                const float ce = !ce_on ? 0.0f
                                 : DUAL ? bad - log_share(xy, M, untempered_ref<POW>(M, u), kLog2e, far, S1)
                                        : bad - lp;
                const float loss = (row_kd ? a.kd_weight * kd : bad) + (ce_on ? a.ce_weight * ce : 0.0f);
                if (out) {
                    if (a.loss) a.loss[r] = loss;
                    sum.loss += loss; sum.first += kd; sum.second += ce; sum.count += 1.0;
                }
            }
            par ^= 1;
            buf4 = (buf4 + 1) & 3;
        }
        if (kGrad && rank == 0) finish_sums(a, sum, group, ngroups);
    } else {
        // ------------------------------------------------------------ the element warps
        const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + 16u * uint32_t(tid);
        auto row_at = [&](int64_t r) { return static_cast<const T*>(a.x) + r * a.ld; };
        // all rows lie alike where their stride is a multiple of 128 bytes
        const bool alike = (a.ld * int(sizeof(T))) % 128 == 0;
        const Place<T> first_place(static_cast<const T*>(a.x), a.vocab, rank, clog);
        auto place_of = [&](const T* x) { return alike ? first_place : Place<T>(x, a.vocab, rank, clog); };
        // Between its passes a share stays in its slot (kept) where it fits a tile, whatever
        // the row's phase; else its tiles are copied again.
        const bool kept = grad && ((a.vocab / N + cluster - 1) >> clog) + (alike ? first_place.off : 7) <= tile;
        const bool again = grad && !kept;
        // The copies run ahead in the order of their use.
        int64_t fr = group - ngroups, fynext = a.target && group < a.rows ? a.target[group] : 0;
        const T *fat = nullptr, *flast = nullptr;   // this thread's next vector, and where row fr's start
        int fleft = 0, nlast = 0;                   // places left of the pass, and those of the row's share
        int foff = 0, flo = 0;                      // empty places before the next vector, and before the row's share
        bool fback = false;                         // the pass is B
        auto segment = [&]() {
            foff = flo;
            if (again && nlast > 0 && !fback) {   // pass B of the row whose pass A is asked for
                fat = flast;
                fleft = nlast;
                fback = true;
                return;
            }
            fback = false;
            nlast = 0;
            while (nlast <= 0) {   // the next row that is not ignored and of which this CTA has a share
                fr += ngroups;
                if (fr >= a.rows) break;
                const int64_t y = fynext;
                if (a.target && fr + ngroups < a.rows) fynext = a.target[fr + ngroups];
                if (y < 0) continue;
                const T* const x = row_at(fr);
                const Place<T> pl = place_of(x);
                foff = flo = pl.off;
                nlast = pl.hi > pl.lo ? pl.hi - pl.lo + pl.off : 0;
                flast = x + pl.head + (pl.lo + tid - pl.off) * N;
            }
            fat = flast;
            fleft = nlast;
        };
        auto issue = [&](int slot) {
            const uint32_t to = ring_at + 16u * uint32_t(slot * tile);
            if (fleft >= tile && foff == 0) {
#pragma unroll
                for (int i = 0; i < kTileVecs; ++i) copy_async(to + 16u * B * i, fat + B * N * i);
            } else {   // behind the last row a group is empty
#pragma unroll
                for (int i = 0; i < kTileVecs; ++i)
                    if (tid + B * i < fleft && (i > 0 || tid >= foff)) copy_async(to + 16u * B * i, fat + B * N * i);
                if (tid < foff)
                    ring[slot * tile + tid] = make_uint4(Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty);
                foff = 0;
            }
            fat += tile * N;
            fleft -= tile;
            copy_commit();
        };
        auto fetch = [&](int slot) {
            if (fleft <= 0) segment();
            issue(slot);
        };
        int slot = -1;   // of the tile last taken
        auto take_tile = [&]() {
            const int before = slot;
            slot = slot + 1 == ST ? 0 : slot + 1;
            if (kept) {
                copy_wait<ST - 2>();
            } else {   // the tile before is done with; its slot is the next to fill
                fetch(before < 0 ? ST - 1 : before);
                copy_wait<ST - 1>();
            }
        };

        // the teacher's entry of this thread for the group's next row
        int64_t nid = -1;
        float nt = 0.0f;
        auto ask_teacher = [&](int64_t r) {
            if (tid < a.k && r < a.rows) {
                nid = teacher_id(a, r * a.ldt + tid);
                nt = teacher_logit(a, r * a.ldt + tid);
            }
        };

        // The teacher's elements of a row, written again over the dense gradient once every warp
        // has stored its part of that: an id's first entry takes the weights of all that are
        // equal to it.  Four lanes to an entry look for equal ids where that keeps all of them
        // busy at once, else one.
        int64_t listed = -1, listed_y = 0;
        int listed_buf = 0;
        auto relist = [&]() {
            const float4 fc = fac[listed_buf][0], f1 = fac[listed_buf][1];
            const float* const tb = teach + listed_buf * 3 * kpad;
            const float Mb = fc.x, kq = fc.y, cq = fc.z, tm = f1.y, tu = f1.z, wp = f1.x;
            const bool tfar = big(tm, c2);
            auto share = [&](int j) {   // the teacher's exponential of entry j
                return ex2(tfar ? (tb[kpad + j] - tm) * c2 : __fmaf_rn(tb[kpad + j], c2, -tu));
            };
            const int n = wp != 0.0f ? a.k : 0;
            const int* const ids = reinterpret_cast<const int*>(tb);
            const Place<T> pl = place_of(row_at(listed));
            T* const dx = static_cast<T*>(a.dx) + listed * a.ldd;
            const int ls = 4 * n <= B ? 2 : 0, part = lane & ((1 << ls) - 1);
            for (int base = (warp * 32) >> ls; base < n; base += B >> ls) {
                const int i = base + (lane >> ls), id = i < n ? ids[i] : -1;
                int same = 0;   // entries of this id
#pragma unroll 2
                for (int j = 4 * part; j < n; j += 4 << ls) {   // ids are padded with -1 to a multiple of 4
                    const int4 q = *reinterpret_cast<const int4*>(ids + j);
                    same += int(q.x == id) + int(q.y == id) + int(q.z == id) + int(q.w == id);
                }
                if (ls != 0) {
                    same += __shfl_xor_sync(~0u, same, 1);
                    same += __shfl_xor_sync(~0u, same, 2);
                }
                bool at_edge;
                int v;
                // the label's element has its value already
                if (part != 0 || id < 0 || (ce_on && id == int(listed_y)) || !pl.owns(id, rank, at_edge, v)) continue;
                float w = 0.0f;
                bool lead = true;
                if (same == 1) {
                    w = wp * share(i);
                } else {
                    for (int j = 0; j < n; ++j) {
                        if (ids[j] != id) continue;
                        lead = lead && j >= i;
                        w = __fmaf_rn(wp, share(j), w);
                    }
                }
                if (lead) dx[id] = from_f<T>(dense_value(tb[2 * kpad + i], Mb, kq, cq) - w);
            }
            listed = -1;
        };

        // pass B of row r: its label, the value of this thread's edge element, its slot (kept)
        auto back = [&](int64_t r, int64_t y, float xe, int kept_slot, int was, int buffer) {
            bar_sync(3 + was, B + 32);   // the row's factors
            if (!grad) return;
            if (kTeach && listed >= 0 && !again) relist();
            const T* const x = row_at(r);
            const Place<T> pl = place_of(x);
            const int lo = pl.lo, hi = pl.hi;
            T* const dx = static_cast<T*>(a.dx) + r * a.ldd;
            const bool whole = same_phase(x, static_cast<const T*>(dx));
            const bool edge = rank == 0 && tid < pl.edges;
            const float4 fc = fac[buffer][0];
            const float Mb = fc.x, kq = fc.y, cq = OP == kDistill ? fc.z : 0.0f;
            const float u = anchor(Mb, c2), v1 = DUAL ? untempered_ref<POW>(Mb, u) : 0.0f;
            auto dense = [&](float x) { return dense_value(x, Mb, kq, cq); };
            for (int done = 0; hi > lo && done < hi - lo + pl.off; done += tile) {
                if (!kept) take_tile();
                const uint4* const buf = ring + (kept ? kept_slot : slot) * tile + tid;
                const int mine = hi - lo + pl.off - done - tid;   // vector i of the thread exists where B i < mine
                const bool none = done == 0 && tid < pl.off;      // but for its first one here
                T* const to = dx + pl.head + (lo + done + tid - pl.off) * N;
                if (big(Mb, c2)) {   // NaN rows too
#pragma unroll 1
                    for (int i = none ? 1 : 0; i < kTileVecs && B * i < mine; ++i)
#pragma unroll 1
                        for (int j = 0; j < N; ++j)
                            to[B * N * i + j] = from_f<T>(dense(to_f(reinterpret_cast<const T*>(buf + B * i)[j])));
                    continue;
                }
                auto emit = [&](int i) {
                    float f[N];
                    Vec<T>::wide(buf[B * i], f);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float e = ex2(__fmaf_rn(f[j], c2, -u));
                        f[j] = DUAL ? mix<POW>(e, f[j], v1, kq, cq) : e * kq;
                    }
                    store_vec<T>(to + B * N * i, Vec<T>::narrow(f), whole);
                };
#pragma unroll 1
                for (int g = 0; g < kTileVecs; g += U) {
                    if (whole && B * (g + U - 1) < mine && (g > 0 || !none)) {
#pragma unroll
                        for (int i = 0; i < U; ++i) emit(g + i);
                    } else {
#pragma unroll 1
                        for (int i = g == 0 && none ? 1 : g; i < g + U && B * i < mine; ++i) emit(i);
                    }
                }
            }
            if (kept && hi > lo) fetch(kept_slot);
            if (edge) dx[pl.edge_at(tid)] = from_f<T>(dense(xe));
            if ((OP == kPolicy || ce_on) && y < a.vocab) {
                // the label's element again, by the thread that stored it
                bool at_edge;
                int v;
                if (pl.owns(int(y), rank, at_edge, v) && (at_edge ? v : (v - lo + pl.off) & (B - 1)) == tid) dx[y] = from_f<T>(fc.w);
            }
            if (kTeach && kd_on) {
                listed = r;
                listed_y = y;
                listed_buf = buffer;
            }
        };

        // The group's first row is taken to count: its first tile is asked for along with its label.
        bool guessed = false;
        if (group < a.rows) {
            const T* const x = row_at(group);
            const Place<T> pl = place_of(x);
            fr = group;
            foff = flo = pl.off;
            nlast = fleft = pl.hi > pl.lo ? pl.hi - pl.lo + pl.off : 0;
            flast = fat = x + pl.head + (pl.lo + tid - pl.off) * N;
            issue(0);
            guessed = fynext >= 0 && nlast > 0;
            if (a.target && group + ngroups < a.rows) fynext = a.target[group + ngroups];
            if (!guessed) {
                copy_wait<0>();
                fleft = nlast = 0;
            }
        }
        if (!guessed) fetch(0);
#pragma unroll
        for (int i = 1; i < ST - 1; ++i) fetch(i);
        if (kept) fetch(ST - 1);
        if (kTeach && kd_on) ask_teacher(group);
        if (cluster > 1) {
            cluster_arrive_relaxed();
            cluster_wait();
        }
        // the row whose pass B is next
        int64_t back_row = -1, back_y = 0;
        float back_xe = 0.0f;
        int back_slot = 0, back_par = 0, back_buf = 0;
        bool exchanged = false;   // some row's parts went to the cluster
        for (int64_t r = group;; r += ngroups) {
            const bool live = r < a.rows;
            int64_t y = 0;
            float xe = kNegInf;
            if (live) {
                y = label(r);
                const T* const x = row_at(r);
                const Place<T> pl = place_of(x);
                const int lo = pl.lo, hi = pl.hi;
                const bool edge = rank == 0 && tid < pl.edges;
                if (y < 0) {
                    if (grad) {
                        T* const dx = static_cast<T*>(a.dx) + r * a.ldd;
                        const bool whole = same_phase(x, static_cast<const T*>(dx));
                        for (int v = lo + tid; v < hi; v += B) store_vec<T>(dx + pl.head + v * N, make_uint4(0, 0, 0, 0), whole);
                        if (edge) dx[pl.edge_at(tid)] = from_f<T>(0.0f);
                    }
                    if (kTeach && kd_on) ask_teacher(r + ngroups);
                    continue;
                }
                if (edge) xe = to_f(x[pl.edge_at(tid)]);
                // the teacher's entry of this thread (asked for a row ago), and the student's logit there
                const int64_t id0 = nid;
                const float t0 = nt;
                float z0 = 0.0f;
                if (kTeach && kd_on) {
                    if (tid < a.k && id0 >= 0 && id0 < a.vocab) z0 = to_f(x[id0]);
                    ask_teacher(r + ngroups);
                }
                // pass A: the thread's reference (its largest element so far, or near it) and its sums, U
                // vectors at a time
                float m = kNegInf, acc = 0.0f, acc1 = 0.0f;
                auto raise = [&](float top) {   // the sums so far to a much larger element
                    // smaller steps are left: m is a reference, and exponentials up to 2^32 of it do no harm
                    if (!((top - m) * (DUAL ? fmaxf(c2, kLog2e) : c2) > 32.0f)) return;
                    acc *= rescale(m, top, c2);
                    if (DUAL) acc1 *= rescale1<POW>(m, top, c2);
                    m = top;
                };
                auto add_big = [&](const uint4* at) {
#pragma unroll 1
                    for (int j = 0; j < N; ++j) {
                        const float x = to_f(reinterpret_cast<const T*>(at)[j]), d = x - part_ref(m);
                        acc += ex2(d * c2);
                        if (DUAL) acc1 += ex2(d * kLog2e);
                    }
                };
                auto add = [&](const uint4 (&raw)[U], float u, float v) {
                    float sum[U], sum1[U];
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        float f[N], e[N];
                        Vec<T>::wide(raw[i], f);
#pragma unroll
                        for (int j = 0; j < N; ++j) e[j] = ex2(__fmaf_rn(f[j], c2, -u));
                        sum[i] = tree_sum(e);
                        if constexpr (DUAL) sum1[i] = untempered_sum<POW>(e, f, v);
                    }
                    acc += tree_sum(sum);
                    if constexpr (DUAL) acc1 += tree_sum(sum1);
                };
                for (int left = hi > lo ? hi - lo + pl.off : 0; left > 0; left -= tile) {
                    take_tile();
                    const uint4* const buf = ring + slot * tile + tid;
                    const int mine = left - tid;
#pragma unroll 1
                    for (int g = 0; g < kTileVecs; g += U) {
                        if (B * g >= mine) break;
                        uint4 raw[U];
                        if (B * (g + U - 1) < mine) {
#pragma unroll
                            for (int i = 0; i < U; ++i) raw[i] = buf[B * (g + i)];
                        } else {
#pragma unroll
                            for (int i = 0; i < U; ++i) {
                                raw[i] = make_uint4(Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty);
                                if (B * (g + i) < mine) raw[i] = buf[B * (g + i)];
                            }
                        }
                        float top = m;
#pragma unroll
                        for (int i = 0; i < U; ++i) top = fmaxf(top, Vec<T>::top(raw[i]));
                        raise(top);
                        if (big(part_ref(m), c2)) {
#pragma unroll 1
                            for (int i = 0; i < U; ++i)
                                if (B * (g + i) < mine) add_big(buf + B * (g + i));
                        } else {
                            const float u = anchor(part_ref(m), c2), u1 = DUAL ? untempered_ref<POW>(part_ref(m), u) : 0.0f;
                            add(raw, u, u1);
                        }
                    }
                }
                {
                    // the warp's part, edges included
                    const float top = warp_max(fmaxf(m, xe)), ref = part_ref(top);
                    const float ee = power(xe, ref, c2);
                    const float s = warp_sum(acc * rescale(m, ref, c2) + ee);
                    float s1 = 0.0f;
                    if (DUAL) s1 = warp_sum(acc1 * rescale1<POW>(m, ref, c2) + power1<POW>(ee, xe, ref, c2));
                    if (lane == 0) wparts[par][warp] = make_float4(top, s, s1, 0.0f);
                }
                if (kTeach && kd_on && warp * 32 < a.k) {
                    // the teacher's largest logit and sums over the warp's entries; the first of each
                    // thread is in registers
                    float* const tb = teach + buf4 * 3 * kpad;
                    if (tid < kpad - a.k) tb[a.k + tid] = __int_as_float(-1);
                    auto entry = [&](int j, int64_t id, float logit, float x) {   // into the buffer; -inf: none
                        const bool on = id >= 0 && id < a.vocab;
                        const float t = on ? logit : kNegInf;
                        tb[j] = __int_as_float(on ? int(id) : -1);
                        tb[kpad + j] = t;
                        tb[2 * kpad + j] = x;
                        return t;
                    };
                    TeacherPart te{kNegInf, 0.0f, 0.0f, 0.0f};
                    bool beyond = tid < a.k && id0 >= a.vocab;
                    if (tid < a.k) {
                        const float t = entry(tid, id0, t0, z0);
                        te = teacher_entry(t, t == kNegInf ? 0.0f : power(t, t, c2), z0);
                    }
                    for (int j = tid + B; j < a.k; j += B) {
                        const int64_t id = teacher_id(a, r * a.ldt + j);
                        const float z = id >= 0 && id < a.vocab ? to_f(x[id]) : 0.0f;
                        const float t = entry(j, id, teacher_logit(a, r * a.ldt + j), z);
                        beyond = beyond || id >= a.vocab;
                        const float m = fmaxf(te.m, t), f = rescale(te.m, part_ref(m), c2);
                        const TeacherPart one = teacher_entry(t, power(t, part_ref(m), c2), z);
                        const float first = te.m > kNegInf && te.d < INFINITY ? te.z : one.z;
                        te = {m, te.s * f + one.s, moved(te, f, m, first) + moved(one, 1.0f, m, first), first};
                    }
                    te = warp_join(te, c2);
                    if (__any_sync(~0u, beyond)) te.s = kNaN;
                    if (lane == 0) tparts[par][warp] = te;
                }
                if (cluster > 1) {
                    if (exchanged) cluster_wait();   // of the row before: long past
                    cluster_arrive_relaxed();
                    exchanged = true;
                }
                if (kTeach && again) {
                    // pass B of this row waits for its factors anyway: meanwhile the row before,
                    // of which every warp has stored its part
                    bar_sync(1 + par, B + 32);
                    if (listed >= 0) relist();
                } else {
                    bar_arrive(1 + par, B + 32);
                }
            }
            if (again && live) {   // not kept waiting: two rows under way would not fit L2
                back_row = r;
                back_y = y;
                back_xe = xe;
                back_par = par;
                back_buf = buf4;
            }
            if (back_row >= 0) back(back_row, back_y, back_xe, back_slot, back_par, back_buf);
            if (!live) break;
            back_row = again ? -1 : r;
            back_y = y;
            back_xe = xe;
            back_slot = slot;
            back_par = par;
            back_buf = buf4;
            par ^= 1;
            buf4 = (buf4 + 1) & 3;
        }
        if (kTeach && listed >= 0) {
            bar_sync(5, B);
            relist();
        }
        if (exchanged) cluster_wait();
        copy_wait<0>();
    }
    if (OP == kPrefStat && rank == 0) finish_pairs<B, B>(a, ngroups);
}

// The same as ex2, taken again: the compiler would keep every exponential of the first pass
// in a register instead (116 to 255 of them).
__device__ __forceinline__ float ex2_again(float v) {
    float r;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Many short rows: a warp per row, the row in its registers (NV vectors per lane; policy with 17
// vectors of 16-bit logits does not fit 128 of them and spills 328 bytes per thread), no barrier
// at all.  What bounds it: instructions, about 300 for a row besides 11 per element, and the
// latency of a row's loads with 16 to 24 warps per SM.  Share of the copy rate on 16,384 bf16
// rows against k_row: policy 37 / 17 % at 1,000 entries, 39 / 25 at 2,001, 65 / 51 at 4,096;
// log-probabilities 36 / 15, 40 / 25, 69 / 45.  Preference's statistics take it too;
// distillation, whose entries want more lanes, does not.
template <typename T, int OP, int NV>
__global__ void __launch_bounds__(256, NV > 4 ? 2 : 3) k_short(const LossArgs a) {
    constexpr int N = Vec<T>::N;
    constexpr bool kGrad = OP == kPolicy;
    if (OP == kPrefStat) asm volatile("griddepcontrol.launch_dependents;");   // the gradient's kernel, see there
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * 8;
    const float c2 = a.it * kLog2e, kNaN = __int_as_float(0x7fffffff);
    const float step = (kGrad && a.seed ? *a.seed : 1.0f) * a.inv_n;
    LossSums sum;
    const int64_t start = int64_t(blockIdx.x) * 8 + warp;
    int64_t ynext = start < a.rows ? a.target[start] : 0;
    for (int64_t r = start; r < a.rows; r += warps) {
        const int64_t y = ynext;
        if (r + warps < a.rows) ynext = a.target[r + warps];
        const T* const x = static_cast<const T*>(a.x) + r * a.ld;
        T* const dx = kGrad && a.dx ? static_cast<T*>(a.dx) + r * a.ldd : nullptr;
        const Place<T> pl(x, a.vocab, 0, 0);
        const bool whole = kGrad && same_phase(x, static_cast<const T*>(dx)), edge = lane < pl.edges;
        const T* const body = x + pl.head;
        if (y < 0) {
            if (dx) {
                for (int v = lane; v < pl.body; v += 32) store_vec<T>(dx + pl.head + v * N, make_uint4(0, 0, 0, 0), whole);
                if (edge) dx[pl.edge_at(lane)] = from_f<T>(0.0f);
            }
            if (lane == 0) {
                if (a.logp) a.logp[r] = 0.0f;
                if (kGrad && a.loss) a.loss[r] = 0.0f;
                if (OP == kPrefStat) a.stat[r] = {0.0f, 0.0f, 0.0f, 0.0f};
            }
            continue;
        }
        uint4 raw[NV];
        float m = kNegInf;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * 32 + lane - pl.off;
            raw[i] = make_uint4(Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty);
            if (v >= 0 && v < pl.body) raw[i] = ld16(body + v * N);
        }
        const float xe = edge ? to_f(x[pl.edge_at(lane)]) : kNegInf, xy = to_f(x[y < a.vocab ? y : 0]);
        float old = 0.0f, adv = 0.0f, refl = 0.0f;
        if (OP == kPolicy) {
            old = a.old_logp[r];
            adv = a.adv[r];
        }
        if (OP != kLogprob) refl = a.ref_logp ? a.ref_logp[r] : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) m = fmaxf(m, Vec<T>::top(raw[i]));
        m = warp_max(fmaxf(m, xe));
        // 2^(x c2 - u), or 2^((x - m) c2) of a big m
        const bool far = big(part_ref(m), c2);
        const float u = anchor(part_ref(m), c2), base = far ? m : 0.0f, off = far ? 0.0f : u;
        float acc[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[N];
            Vec<T>::wide(raw[i], f);
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j & 1] += ex2(__fmaf_rn(f[j] - base, c2, -off));
        }
        const float S = warp_sum(acc[0] + acc[1] + ex2(__fmaf_rn(xe - base, c2, -off)));
        const float bad = y >= a.vocab || m == kNegInf ? kNaN : 0.0f;
        const float lp = log_share(xy, m, u, c2, far, S) + bad;
        if (lane == 0 && a.logp) a.logp[r] = lp;
        if (OP == kPrefStat && lane == 0) a.stat[r] = {m + bad, 1.0f / S, 0.0f, lp - refl};
        if (OP != kPolicy) continue;
        float loss, sur, kl;
        const float w = policy_row(a, lp, old, adv, refl, loss, sur, kl) * step * a.it, kq = -w / S;
        if (lane == 0) {
            if (a.loss) a.loss[r] = loss;
            sum.loss += loss; sum.first += sur; sum.second += kl; sum.count += 1.0;
        }
        if (!dx) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * 32 + lane - pl.off;
            if (v >= 0 && v < pl.body) {
                float f[N];
                Vec<T>::wide(raw[i], f);
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] = ex2_again(__fmaf_rn(f[j] - base, c2, -off)) * kq;
                store_vec<T>(dx + pl.head + v * N, Vec<T>::narrow(f), whole);
            }
        }
        if (edge) dx[pl.edge_at(lane)] = from_f<T>(ex2(__fmaf_rn(xe - base, c2, -off)) * kq);
        if (y < a.vocab) {   // the label's element again, by the lane that stored it
            bool at_edge;
            int v;
            pl.owns(int(y), 0, at_edge, v);
            if ((at_edge ? v : (v + pl.off) & 31) == lane)
                dx[y] = from_f<T>(__fmaf_rn(ex2(__fmaf_rn(xy - base, c2, -off)), kq, w));
        }
    }
    if (OP == kPrefStat) finish_pairs<256, 0>(a, int(gridDim.x));
    if (OP == kPolicy) {
        __shared__ LossSums sums[8];
        if (lane == 0) sums[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            if (lane == 0)
                for (int w = 1; w < 8; ++w) {
                    sum.loss += sums[w].loss; sum.first += sums[w].first;
                    sum.second += sums[w].second; sum.count += sums[w].count;
                }
            finish_sums(a, sum, int(blockIdx.x), int(gridDim.x));
        }
    }
}

// Second preference pass: every element from its row's statistics (the pair's derivative
// needs whole sequences first), one segment of a row per CTA, the last rows first (the first
// pass left them in L2).  4,096 x 128,256 bf16, a quarter ignored: 255 us for 1.84 GB.  It is launched to start
// while the first pass runs: its CTAs read their part of the logits, and wait for that
// kernel's end before they use the statistics.
template <typename T, int NV, int TB>
__global__ void __launch_bounds__(TB) k_pref_grad(const LossArgs a, const int segs) {
    constexpr int N = Vec<T>::N;
    const int tid = threadIdx.x;
    const int64_t item = int64_t(gridDim.x) - 1 - blockIdx.x, r = item / segs;
    const int seg = int(item - r * segs);
    const T* const x = static_cast<const T*>(a.x) + r * a.ld;
    const Place<T> row(x, a.vocab, 0, 0);
    T* dx = static_cast<T*>(a.dx) + r * a.ldd;
    const bool whole = same_phase(x, static_cast<const T*>(dx));
    const T* body = x + row.head;
    // segments end on 128-byte boundaries: the first one is short by `off` vectors
    const int lo = seg * NV * TB - row.off, hi = min(row.body, lo + NV * TB);
    const int64_t y = a.target[r];
    const bool edge = seg == 0 && tid < row.edges;
    auto zeros = [&]() {
        for (int v = lo + tid; v < hi; v += TB)
            if (v >= 0) store_vec<T>(dx + row.head + int64_t(v) * N, make_uint4(0, 0, 0, 0), whole);
        if (edge) dx[row.edge_at(tid)] = from_f<T>(0.0f);
    };
    // every CTA waits for the first pass, so that this grid does not end before it
    auto first_pass = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
    if (y < 0) {   // ignored: the first pass does not look at the row
        zeros();
        first_pass();
        return;
    }
    uint4 raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lo + i * TB + tid;
        if (v >= 0 && v < hi) raw[i] = ld16(body + int64_t(v) * N);
    }
    const float xe = edge ? to_f(x[row.edge_at(tid)]) : 0.0f;
    // the label's element: its thread stores it after its vector
    int mine = -1;
    float xy = 0.0f;
    if (y < a.vocab) {
        const int j = int(y), v = (j - row.head) / N;
        const bool at_edge = j < row.head || v >= row.body;
        if (at_edge ? edge && row.edge_at(tid) == j : v >= lo && v < hi && (v - lo) % TB == tid) {
            mine = j;
            xy = to_f(x[j]);
        }
    }
    // everything so far was input; the statistics are the first pass's, which may still be running
    first_pass();
    const RowStat st = a.stat[r];
    if (st.w == 0.0f) {   // outside every sequence, or of a saturated pair
        zeros();
        return;
    }
    const float c2 = a.it * kLog2e, kq = -st.w * st.rs, u = anchor(st.m, c2);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lo + i * TB + tid;
        if (v >= 0 && v < hi) {
            float f[N];
            Vec<T>::wide(raw[i], f);
            if (big(st.m, c2)) {
                for (int j = 0; j < N; ++j) f[j] = ex2((f[j] - st.m) * c2) * kq;
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] = ex2(__fmaf_rn(f[j], c2, -u)) * kq;
            }
            store_vec<T>(dx + row.head + int64_t(v) * N, Vec<T>::narrow(f), whole);
        }
    }
    if (edge) dx[row.edge_at(tid)] = from_f<T>(power(xe, st.m, c2) * kq);
    if (mine >= 0) dx[mine] = from_f<T>(__fmaf_rn(power(xy, st.m, c2), kq, st.w));
}

template <typename T>
RowShape shape_for(int op, int64_t rows, int vocab, bool grad, int sms) {
    const int vecs = (vocab + Vec<T>::N - 1) / Vec<T>::N;
    RowShape s{64, 0};
    // Threads: more where a row is long enough to keep them busy.  Share of the copy rate on
    // thousands of bf16 rows with 64 / 128 / 256 threads: policy 58 / 55 / 31 % at 4,096
    // entries, 64 / 80 / 59 at 8,192, 73 / 83 / 74 at 24,000, 77 / 77 / 88 at 32,768;
    // log-probabilities 82 / 95 / 85 at 32,768, 89 / 93 / 97 at 80,000; distillation
    // 56 / 70 / 58 at 32,768, 58 / 61 / 74 at 80,000.
    if (vecs >= 512) s.threads = vecs > (op == kPolicy && grad ? 3500 : 8192) ? 256 : 128;
    // Long rows are read twice, the second time out of L2 if what is under way (two CTAs per
    // SM) fits it: more CTAs to a row where it would not.
    const int64_t under_way = int64_t(2) * sms * vocab * int(sizeof(T));
    if (grad && s.threads == 256) {
        // 1,824 rows of 80,000 (49 MB): 75 % of the copy rate with 1 CTA per row, 76 with 2;
        // 1,216 of 128,256 (78 MB): 67 with 1, 85 with 2; 2,432 of 50,000 (30 MB): 79 with 1, 58 with 2
        while (s.clog < kMaxClusterLog && under_way >> s.clog > kRowsInL2) s.clog += 1;
    }
    // few rows: spread each over more CTAs while the GPU has idle SMs and the share is over a tile
    while (s.clog < kMaxClusterLog && rows << (s.clog + 1) <= sms && (s.threads * kTileVecs) << s.clog < vecs) s.clog += 1;
    return s;
}

// Row groups that a launch can have resident at once, from the context's cache.
cudaError_t resident_groups(const void* kernel, const cudaLaunchConfig_t& cfg, const RowShape& sh, int sms,
                            GroupCache& cache, int& groups) {
    const int smem = int(cfg.dynamicSmemBytes);
    for (int i = 0; i < cache.n; ++i) {
        const GroupCache::Entry& e = cache.v[i];
        if (e.kernel == kernel && e.threads == sh.threads && e.cluster == sh.clog && e.smem == smem) {
            groups = e.groups;
            return cudaSuccess;
        }
    }
    // one limit for every shape of the kernel: the attribute belongs to the function
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRingBytes);
    if (e != cudaSuccess) return e;
    if (sh.clog > 0) {
        e = cudaOccupancyMaxActiveClusters(&groups, kernel, &cfg);
    } else {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&groups, kernel, int(cfg.blockDim.x), cfg.dynamicSmemBytes);
        groups *= sms;
    }
    if (e != cudaSuccess) return e;
    groups = groups < 1 ? 1 : groups > kMaxLossClusters ? kMaxLossClusters : groups;
    cache.v[cache.n % GroupCache::kEntries] = {kernel, sh.threads, sh.clog, smem, groups};
    if (cache.n < GroupCache::kEntries) cache.n += 1;
    return cudaSuccess;
}

template <typename T, int OP, int B, int POW>
cudaError_t row_launch(const LossArgs& a, const RowShape& sh, int sms, GroupCache& cache, cudaStream_t s) {
    auto* kernel = k_row<T, OP, B, POW>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1u << sh.clog);
    cfg.blockDim = dim3(unsigned(B + 32));
    cfg.dynamicSmemBytes = size_t(16) * kStages * kTileVecs * B + (OP == kDistill ? sizeof(float) * 4 * 3 * size_t((a.k + 63) / 64 * 64) : 0);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << sh.clog;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = sh.clog > 0 ? 1 : 0;
    int groups = 0;
    cudaError_t e = resident_groups(reinterpret_cast<const void*>(kernel), cfg, sh, sms, cache, groups);
    if (e != cudaSuccess) return e;
    if (groups > a.rows) groups = a.rows < 1 ? 1 : int(a.rows);
    cfg.gridDim.x = unsigned(groups) << sh.clog;
    return cudaLaunchKernelEx(&cfg, kernel, a, int(sh.clog));
}

template <typename T, int OP, int POW = kSingle>
cudaError_t rows_by_threads(const LossArgs& a, const RowShape& sh, int sms, GroupCache& cache, cudaStream_t s) {
    if (sh.threads == 64) return row_launch<T, OP, 64, POW>(a, sh, sms, cache, s);
    if (sh.threads == 128) return row_launch<T, OP, 128, POW>(a, sh, sms, cache, s);
    return row_launch<T, OP, 256, POW>(a, sh, sms, cache, s);
}

// Rows of up to 32 NV places, where there are enough of them for a warp each: from kShortRows
// on with NV 4 and 8, from kLongerRows on with NV 17.  us of k_short / k_row, bf16 policy:
// 1,000 entries 7.1 / 6.7 with 128 rows, 7.1 / 7.7 with 256, 7.5 / 11.8 with 1,024; 4,096 entries
// 9.7 / 7.8 with 256 rows, 10.4 / 10.0 with 512, 10.6 / 12.2 with 768; f32 policy of 2,001 entries
// 7.9 / 7.8 with 256 rows, 8.2 / 9.7 with 512; fp16 preference, gradient and all, of 1,000 entries
// 9.5 / 14.7 with 256 rows, of 4,096 entries 10.9 / 13.4 with 512.
constexpr int64_t kShortRows = 256, kLongerRows = 512;

template <typename T, int OP, int NV>
cudaError_t short_launch(const LossArgs& a, int sms, GroupCache& cache, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    auto* kernel = k_short<T, OP, NV>;
    int groups = 0;
    cudaError_t e = resident_groups(reinterpret_cast<const void*>(kernel), cfg, RowShape{256, 0}, sms, cache, groups);
    if (e != cudaSuccess) return e;
    const int64_t want = (a.rows + 7) / 8;
    cfg.gridDim.x = unsigned(groups < want ? groups : want);
    return cudaLaunchKernelEx(&cfg, kernel, a);
}
template <typename T, int OP>
cudaError_t rows_by_length(const LossArgs& a, const RowShape& sh, int sms, GroupCache& cache, cudaStream_t s) {
    const int places = (a.vocab + Vec<T>::N - 1) / Vec<T>::N + 7;
    if (a.rows >= kShortRows && places <= 32 * 4) return short_launch<T, OP, 4>(a, sms, cache, s);
    if (a.rows >= kShortRows && places <= 32 * 8) return short_launch<T, OP, 8>(a, sms, cache, s);
    if (a.rows >= kLongerRows && places <= 32 * 17) return short_launch<T, OP, 17>(a, sms, cache, s);
    return rows_by_threads<T, OP>(a, sh, sms, cache, s);
}

template <typename T>
cudaError_t rows_by_op(int op, const LossArgs& a, int sms, GroupCache& cache, cudaStream_t s) {
    const bool grad = a.dx != nullptr && (op == kPolicy || op == kDistill);
    const RowShape sh = shape_for<T>(op, a.rows, a.vocab, grad, sms);
    switch (op) {
        case kLogprob: return rows_by_length<T, kLogprob>(a, sh, sms, cache, s);
        case kPolicy: return rows_by_length<T, kPolicy>(a, sh, sms, cache, s);
        case kPrefStat: return rows_by_length<T, kPrefStat>(a, sh, sms, cache, s);
        default: break;
    }
    if (a.k == 0 || a.ce_weight == 0.0f || a.it == 1.0f) return rows_by_threads<T, kDistill>(a, sh, sms, cache, s);
    if (a.it == 0.5f) return rows_by_threads<T, kDistill, 2>(a, sh, sms, cache, s);
    if (a.it == 0.25f) return rows_by_threads<T, kDistill, 4>(a, sh, sms, cache, s);
    return rows_by_threads<T, kDistill, 0>(a, sh, sms, cache, s);
}

template <typename T, int TB>
cudaError_t pref_grad_by(const LossArgs& a, cudaStream_t s) {
    constexpr int NV = 4;
    const int vecs = (a.vocab + Vec<T>::N - 1) / Vec<T>::N;
    const int64_t segs = (vecs + 7 + NV * TB - 1) / (NV * TB);
    if (a.rows * segs > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(a.rows * segs));
    cfg.blockDim = dim3(TB);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // starts while the first pass runs
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_pref_grad<T, NV, TB>, a, int(segs));
}
// A CTA no larger than a short row's vectors.
template <typename T>
cudaError_t pref_grad(const LossArgs& a, cudaStream_t s) {
    const int places = (a.vocab + Vec<T>::N - 1) / Vec<T>::N + 7;
    if (places <= 4 * 64) return pref_grad_by<T, 64>(a, s);
    return places <= 4 * 128 ? pref_grad_by<T, 128>(a, s) : pref_grad_by<T, 256>(a, s);
}

}  // namespace

cudaError_t launch_loss_rows(int op, int dt, const LossArgs& a, int sm_count, GroupCache& cache, cudaStream_t s) {
    if (dt == kF32) return rows_by_op<float>(op, a, sm_count, cache, s);
    if (dt == kBF16) return rows_by_op<__nv_bfloat16>(op, a, sm_count, cache, s);
    return rows_by_op<__half>(op, a, sm_count, cache, s);
}

cudaError_t launch_pref_grad(int dt, const LossArgs& a, cudaStream_t s) {
    if (dt == kF32) return pref_grad<float>(a, s);
    if (dt == kBF16) return pref_grad<__nv_bfloat16>(a, s);
    return pref_grad<__half>(a, s);
}

}  // namespace tl
