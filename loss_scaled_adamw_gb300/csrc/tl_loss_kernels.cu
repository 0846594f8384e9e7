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

// A part of a row (a warp's elements) has its largest element m and its sum s of
// exp((x - m) it).  A part without an element above -inf takes 0 in the place of m,
// so its s is 0 (NaN if it holds a NaN), and parts join without -inf - -inf.
__device__ __forceinline__ float part_ref(float m) { return m == kNegInf ? 0.0f : m; }
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

typedef unsigned long long f2;   // two fp32 lanes of the packed instructions
__device__ __forceinline__ f2 pk(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpk(f2 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) { f2 r; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) { f2 r; asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) { f2 r; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c)); return r; }
__device__ __forceinline__ f2 ex2x2(f2 v) {
    float lo, hi;
    unpk(v, lo, hi);
    return pk(ex2(lo), ex2(hi));
}

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
    static __device__ __forceinline__ void wide(uint4 v, f2 (&f)[2]) {
        f[0] = pk(__uint_as_float(v.x), __uint_as_float(v.y));
        f[1] = pk(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ uint4 narrow(const f2 (&f)[2]) {
        float a, b, c, d;
        unpk(f[0], a, b);
        unpk(f[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
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
    static __device__ __forceinline__ f2 one(uint32_t v) { return pk(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }
    static __device__ __forceinline__ void wide(uint4 v, f2 (&f)[4]) { f[0] = one(v.x); f[1] = one(v.y); f[2] = one(v.z); f[3] = one(v.w); }
    static __device__ __forceinline__ uint32_t back(f2 f) {
        float lo, hi;
        unpk(f, lo, hi);
        const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ uint4 narrow(const f2 (&f)[4]) { return make_uint4(back(f[0]), back(f[1]), back(f[2]), back(f[3])); }
};
template <> struct Vec<__half> {
    static constexpr int N = 8;
    static constexpr uint32_t kEmpty = 0xfc00fc00u;
    static __device__ __forceinline__ __half2 h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
    static __device__ __forceinline__ float top(uint4 v) {
        const __half2 m = __hmax2(__hmax2(h2(v.x), h2(v.y)), __hmax2(h2(v.z), h2(v.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ f2 one(uint32_t v) {
        const float2 w = __half22float2(h2(v));
        return pk(w.x, w.y);
    }
    static __device__ __forceinline__ void wide(uint4 v, f2 (&f)[4]) { f[0] = one(v.x); f[1] = one(v.y); f[2] = one(v.z); f[3] = one(v.w); }
    static __device__ __forceinline__ uint32_t back(f2 f) {
        float lo, hi;
        unpk(f, lo, hi);
        const __half2 r = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ uint4 narrow(const f2 (&f)[4]) { return make_uint4(back(f[0]), back(f[1]), back(f[2]), back(f[3])); }
};

// Where a row's elements lie: `head` elements up to the first 16-byte boundary, `body`
// whole vectors from there, and a tail; the head and tail elements ("edges", fewer than
// 2 N) are held one per thread by the first CTA of the group.
template <typename T> struct Row {
    const T* x;
    int head, body, edges;
    __device__ __forceinline__ Row(const T* p, int vocab) : x(p) {
        constexpr int N = Vec<T>::N;
        const int ph = int((reinterpret_cast<uintptr_t>(p) / sizeof(T)) % N);
        head = ph == 0 ? 0 : min(N - ph, vocab);
        body = (vocab - head) / N;
        edges = vocab - body * N;
    }
    __device__ __forceinline__ int edge_at(int i) const { return i < head ? i : i + body * Vec<T>::N; }
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

constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = 16;   // 512 threads

__device__ __forceinline__ uint32_t cluster_rank() { uint32_t r; asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r)); return r; }
__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
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

// e^tau of the temperature's exponential for the cross-entropy at temperature 1: tau = 2,
// 3, 4 by products, else (0) from the logit.
__device__ __forceinline__ f2 untempered(f2 e, f2 d, int pow) {
    if (pow == 0) return ex2x2(mul2(d, pk(kLog2e, kLog2e)));
    f2 r = mul2(e, e);
    if (pow == 3) r = mul2(r, e);
    if (pow == 4) r = mul2(r, r);
    return r;
}

// One row at a time per group of `cluster` CTAs, each holding a contiguous share of the
// row's vectors in registers (NV per thread): the row is read once.  A warp finds the
// largest of its elements and their sum, writes both into every CTA of the group
// (distributed shared memory), and after one barrier every warp joins all parts and
// goes on to the gradient of the elements that it still holds.  Rows longer than the
// group's registers run in rounds and are read a second time for the gradient.
// DUAL: distillation with both terms at temperatures that differ, two sums per row.
template <typename T, int OP, int NV, bool DUAL>
__global__ void __launch_bounds__(512, 2) k_row(const LossArgs a, const int cluster, const int pow) {
    constexpr int N = Vec<T>::N;
    constexpr bool kTeach = OP == kDistill;
    constexpr bool kGrad = OP == kPolicy || OP == kDistill;
    __shared__ float4 parts[2][kMaxCluster * kMaxWarps];          // m, s, s at temperature 1
    __shared__ float4 tparts[kTeach ? 2 : 1][kMaxWarps];           // teacher: m, sum e, sum e (t - z), bad
    __shared__ float4 rowin[2];                                  // x_y, old, advantage, ref
    extern __shared__ float teach[];                             // [2][k + 1] of id, t / tau, x
    const int B = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = B >> 5;
    const int rank = cluster > 1 ? int(cluster_rank()) : 0;
    const int group = int(blockIdx.x) / cluster, ngroups = int(gridDim.x) / cluster;
    const float c2 = a.it * kLog2e;
    const float step = (a.seed ? *a.seed : 1.0f) * a.inv_n;
    const bool kd_on = kTeach && a.k > 0, ce_on = kTeach && a.ce_weight > 0.0f;
    const float kNaN = __int_as_float(0x7fffffff);
    LossSums sum;
    int par = 0;
    if (cluster > 1) cluster_barrier();   // every CTA of the group runs before any writes into another
    for (int64_t r = group; r < a.rows; r += ngroups) {
        const Row<T> row(static_cast<const T*>(a.x) + r * a.ld, a.vocab);
        T* dx = kGrad && a.dx ? static_cast<T*>(a.dx) + r * a.ldd : nullptr;
        const bool whole = kGrad && same_phase(row.x, static_cast<const T*>(dx));
        const T* body = row.x + row.head;
        const int share = (row.body + cluster - 1) / cluster;
        const int lo = min(row.body, rank * share), hi = min(row.body, lo + share);
        const int64_t y = a.target ? a.target[r] : 0;
        const bool edge = rank == 0 && tid < row.edges;
        if (y < 0) {
            if (dx) {
                for (int v = lo + tid; v < hi; v += B) store_vec<T>(dx + row.head + v * N, make_uint4(0, 0, 0, 0), whole);
                if (edge) dx[row.edge_at(tid)] = from_f<T>(0.0f);
            }
            if (rank == 0 && tid == 0) {
                if (OP != kDistill && a.logp) a.logp[r] = 0.0f;
                if (kGrad && a.loss) a.loss[r] = 0.0f;
                if (OP == kPrefStat) a.stat[r] = {0.0f, 0.0f, 0.0f, 0.0f};
            }
            continue;
        }
        // the row's vectors, all loads under way before the first is used
        uint4 raw[NV];
        float m = kNegInf, s = 0.0f, s1 = 0.0f, xe = kNegInf;
        if (edge) xe = to_f(row.x[row.edge_at(tid)]);
        const int rounds = hi - lo > NV * B ? (hi - lo + NV * B - 1) / (NV * B) : 1;
        if (tid == 0) {
            float4 in;
            in.x = to_f(row.x[y < a.vocab ? y : 0]);
            if (OP == kPolicy) {
                in.y = a.old_logp[r];
                in.z = a.adv[r];
                in.w = a.ref_logp ? a.ref_logp[r] : 0.0f;
            }
            if (OP == kPrefStat) in.w = a.ref_logp ? a.ref_logp[r] : 0.0f;
            rowin[par] = in;
        }
        for (int q = 0; q < rounds; ++q) {
            const int base = lo + q * NV * B;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = base + i * B + tid;
                raw[i] = make_uint4(Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty);
                if (v < hi) raw[i] = ld16(body + int64_t(v) * N);
            }
            if (kTeach && q == 0 && kd_on) {
                // the teacher's entries, a few per thread: logit, id, and the student's logit there
                float* const tb = teach + par * 3 * (a.k + 1);
                float tm = kNegInf, ts = 0.0f, td = 0.0f, bad = 0.0f;
                for (int i = tid; i < a.k; i += B) {
                    const int64_t id = teacher_id(a, r * a.ldt + i);
                    const bool on = id >= 0 && id < a.vocab;
                    const float t = on ? teacher_logit(a, r * a.ldt + i) * a.it : kNegInf;
                    const float z = on ? to_f(row.x[id]) : 0.0f;
                    if (id >= a.vocab) bad = kNaN;
                    tb[i] = __int_as_float(on ? int(id) : -1);
                    tb[a.k + 1 + i] = t;
                    tb[2 * (a.k + 1) + i] = z;
                    // running form: the entries of one thread are few
                    const float nm = fmaxf(tm, t), nr = part_ref(nm);
                    const float f = ex2((part_ref(tm) - nr) * kLog2e);
                    const float e = ex2((t - nr) * kLog2e);
                    ts = (tm == kNegInf ? ts : ts * f) + e;
                    td = (tm == kNegInf ? td : f != 0.0f ? td * f : 0.0f) + (e != 0.0f ? e * (t - z * a.it) : 0.0f);
                    tm = nm;
                }
                const float wm = warp_max(tm), wr = part_ref(wm);
                const float f = tm == kNegInf ? 1.0f : ex2((tm - wr) * kLog2e);
                ts = warp_sum(ts * f);
                td = warp_sum(f != 0.0f ? td * f : 0.0f);
                bad = warp_sum(bad);
                if (lane == 0) tparts[par][warp] = make_float4(wm, ts, td, bad);
            }
            // the warp's largest element; sums of earlier rounds are brought to it
            float top = q == 0 ? xe : kNegInf;
#pragma unroll
            for (int i = 0; i < NV; ++i) top = fmaxf(top, Vec<T>::top(raw[i]));
            top = fmaxf(m, warp_max(top));
            const float ref = part_ref(top);
            if (q > 0) {
                const float d = part_ref(m) - ref;
                if (m != kNegInf) {
                    s *= ex2(d * c2);
                    if (DUAL) s1 *= ex2(d * kLog2e);
                }
            } else {
                const float d = xe - ref, e = ex2(d * c2);
                s = e;
                if (DUAL) { float u, w; unpk(untempered(pk(e, 0.0f), pk(d, 0.0f), pow), u, w); s1 = u; }
            }
            m = top;
            const f2 nref = pk(-ref, -ref), cc = pk(c2, c2);
            f2 acc[2] = {pk(s, 0.0f), pk(0.0f, 0.0f)}, acc1[2] = {pk(s1, 0.0f), pk(0.0f, 0.0f)};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (base + i * B >= hi) break;   // the whole CTA has no vector left
                f2 f[N / 2];
                Vec<T>::wide(raw[i], f);
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    const f2 d = add2(f[j], nref), e = ex2x2(mul2(d, cc));
                    acc[j & 1] = add2(acc[j & 1], e);
                    if (DUAL) acc1[j & 1] = add2(acc1[j & 1], untempered(e, d, pow));
                }
            }
            float u, w;
            unpk(add2(acc[0], acc[1]), u, w);
            s = u + w;
            if (DUAL) {
                unpk(add2(acc1[0], acc1[1]), u, w);
                s1 = u + w;
            }
        }
        s = warp_sum(s);
        if (DUAL) s1 = warp_sum(s1);
        if (cluster > 1) {
            if (lane < cluster) store_remote(&parts[par][rank * nw + warp], uint32_t(lane), make_float4(m, s, s1, 0.0f));
            cluster_barrier();
        } else {
            if (lane == 0) parts[par][warp] = make_float4(m, s, s1, 0.0f);
            __syncthreads();
        }
        // every warp joins the parts of the whole row, in one order
        float S = 0.0f, S1 = 0.0f, M = kNegInf;
        const int np = cluster * nw;
        for (int i = lane; i < np; i += 32) M = fmaxf(M, parts[par][i].x);
        M = warp_max(M);
        const float R = part_ref(M);
        for (int i = lane; i < np; i += 32) {
            const float4 p = parts[par][i];
            const float d = part_ref(p.x) - R;
            S = __fmaf_rn(p.y, p.x == kNegInf ? 1.0f : ex2(d * c2), S);
            if (DUAL) S1 = __fmaf_rn(p.z, p.x == kNegInf ? 1.0f : ex2(d * kLog2e), S1);
        }
        S = warp_sum(S);
        if (DUAL) S1 = warp_sum(S1);
        const float4 in = rowin[par];
        float bad = y >= a.vocab || M == kNegInf ? kNaN : 0.0f;
        const float lg = log2f(S);
        const float lp = __fmaf_rn(in.x - M, c2, -lg) * kLn2 + bad;
        if (OP == kLogprob || OP == kPrefStat) {
            if (rank == 0 && tid == 0) {
                if (a.logp) a.logp[r] = lp;
                if (OP == kPrefStat) a.stat[r] = {M + bad, 1.0f / S, 0.0f, lp - in.w};
            }
        } else {
            float w = 0.0f, kq, cq = 0.0f, wc = 0.0f;   // gradient factors: label, q at the temperature, q at 1
            float tm = kNegInf, ts = 0.0f, td = 0.0f;
            bool row_kd = false;
            if (OP == kPolicy) {
                float loss, sur, kl;
                w = policy_row(a, lp, in.y, in.z, in.w, loss, sur, kl) * step * a.it;
                kq = -w / S;
                if (rank == 0 && tid == 0) {
                    if (a.logp) a.logp[r] = lp;
                    if (a.loss) a.loss[r] = loss;
                    sum.loss += loss; sum.first += sur; sum.second += kl; sum.count += 1.0;
                }
            } else {
                if (kd_on) {
                    const float4 p = lane < nw ? tparts[par][lane] : make_float4(kNegInf, 0.0f, 0.0f, 0.0f);
                    tm = warp_max(p.x);
                    const float f = p.x == kNegInf ? 1.0f : ex2((p.x - part_ref(tm)) * kLog2e);
                    ts = warp_sum(p.y * f);
                    td = warp_sum(f != 0.0f ? p.z * f : 0.0f);
                    bad += warp_sum(p.w);
                    row_kd = ts != 0.0f;
                }
                const float lz = __fmaf_rn(M, a.it, lg * kLn2);   // log sum exp z
                const float kd = row_kd ? (td / ts - tm - logf(ts) + lz) / (a.it * a.it) + bad : bad;
                const float ce = ce_on ? (DUAL ? logf(S1) - (in.x - M) : -lp) + bad : 0.0f;
                const float loss = (row_kd ? a.kd_weight * kd : bad) + (ce_on ? a.ce_weight * ce : 0.0f);
                if (rank == 0 && tid == 0) {
                    if (a.loss) a.loss[r] = loss;
                    sum.loss += loss; sum.first += kd; sum.second += ce; sum.count += 1.0;
                }
                kq = row_kd ? a.kd_weight * step / a.it / S : 0.0f;
                wc = ce_on ? a.ce_weight * step : 0.0f;
                if (DUAL) cq = wc / S1; else kq += wc / S;
                kq += bad;
            }
            if (dx) {
                const float Mb = M + bad;
                const f2 nref = pk(-Mb, -Mb), cc = pk(c2, c2), k2 = pk(kq, kq), k1 = pk(cq, cq);
                for (int q = 0; q < rounds; ++q) {
                    const int base = lo + q * NV * B;
                    if (rounds > 1) {
#pragma unroll
                        for (int i = 0; i < NV; ++i) {
                            const int v = base + i * B + tid;
                            if (v < hi) raw[i] = ld16(body + int64_t(v) * N);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int v = base + i * B + tid;
                        if (v < hi) {
                            f2 f[N / 2];
                            Vec<T>::wide(raw[i], f);
#pragma unroll
                            for (int j = 0; j < N / 2; ++j) {
                                const f2 d = add2(f[j], nref), e = ex2x2(mul2(d, cc));
                                f[j] = DUAL ? fma2(untempered(e, d, pow), k1, mul2(e, k2)) : mul2(e, k2);
                            }
                            store_vec<T>(dx + row.head + int64_t(v) * N, Vec<T>::narrow(f), whole);
                        }
                    }
                }
                auto dense = [&](float x) {
                    const float d = x - Mb, e = ex2(d * c2);
                    float u = 0.0f, t;
                    if (DUAL) unpk(untempered(pk(e, 0.0f), pk(d, 0.0f), pow), u, t);
                    return DUAL ? __fmaf_rn(u, cq, e * kq) : e * kq;
                };
                // who holds element j: the edges' threads of the first CTA, else the share
                auto owned = [&](int j, int& holder) {
                    const int v = (j - row.head) / N;
                    if (j < row.head || v >= row.body) {
                        holder = j < row.head ? j : j - row.body * N;
                        return rank == 0;
                    }
                    holder = (v - lo) % B;
                    return v >= lo && v < hi;
                };
                if (edge) dx[row.edge_at(tid)] = from_f<T>(dense(xe));
                if (OP == kPolicy) {
                    // the label's element again, by the thread that stored it
                    int holder;
                    if (bad == 0.0f && owned(int(y), holder) && holder == tid) dx[y] = from_f<T>(w + dense(in.x));
                } else {
                    // the listed elements again, once the CTA has stored its share: an id's first
                    // entry takes the weights of all that are equal to it
                    const int n = row_kd ? a.k : 0, entries = n + (ce_on && bad == 0.0f ? 1 : 0);
                    const float* const tb = teach + par * 3 * (a.k + 1);
                    const float wp = row_kd ? a.kd_weight * step / (a.it * ts) : 0.0f;
                    __syncthreads();
                    for (int i = tid; i < entries; i += B) {
                        const int id = i < n ? __float_as_int(tb[i]) : int(y);
                        int holder;
                        if (id < 0 || !owned(id, holder)) continue;
                        float v = ce_on && id == int(y) ? wc : 0.0f;
                        bool first = true;
                        for (int j = 0; j < n; ++j) {
                            if (__float_as_int(tb[j]) != id) continue;
                            if (j < i) { first = false; break; }
                            v = __fmaf_rn(wp, ex2((tb[a.k + 1 + j] - tm) * kLog2e), v);
                        }
                        if (first) dx[id] = from_f<T>(dense(i < n ? tb[2 * (a.k + 1) + i] : in.x) - v);
                    }
                }
            }
        }
        par ^= 1;
    }
    if (OP != kLogprob && rank == 0) finish<OP>(a, sum, group, ngroups);
}

// Second preference pass: every element from its row's statistics, one segment of a row
// per CTA, the last rows first (the first pass left them in L2).
template <typename T, int NV>
__global__ void __launch_bounds__(256) k_pref_grad(const LossArgs a, const int segs) {
    constexpr int N = Vec<T>::N;
    const int tid = threadIdx.x;
    const int64_t item = int64_t(gridDim.x) - 1 - blockIdx.x, r = item / segs;
    const int seg = int(item - r * segs);
    const Row<T> row(static_cast<const T*>(a.x) + r * a.ld, a.vocab);
    T* dx = static_cast<T*>(a.dx) + r * a.ldd;
    const bool whole = same_phase(row.x, static_cast<const T*>(dx));
    const T* body = row.x + row.head;
    const int lo = seg * NV * 256, hi = min(row.body, lo + NV * 256);
    const RowStat st = a.stat[r];
    const int64_t y = a.target[r];
    const bool edge = seg == 0 && tid < row.edges;
    if (y < 0 || st.w == 0.0f) {   // ignored, outside every sequence, or a saturated pair
        for (int v = lo + tid; v < hi; v += 256) store_vec<T>(dx + row.head + int64_t(v) * N, make_uint4(0, 0, 0, 0), whole);
        if (edge) dx[row.edge_at(tid)] = from_f<T>(0.0f);
        return;
    }
    uint4 raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lo + i * 256 + tid;
        if (v < hi) raw[i] = ld16(body + int64_t(v) * N);
    }
    const float xe = edge ? to_f(row.x[row.edge_at(tid)]) : 0.0f;
    const float c2 = a.it * kLog2e, kq = -st.w * st.rs;
    // the label's element: its thread stores it after its vector
    int mine = -1;
    float xy = 0.0f;
    if (y < a.vocab) {
        const int j = int(y), v = (j - row.head) / N;
        const bool at_edge = j < row.head || v >= row.body;
        if (at_edge ? edge && row.edge_at(tid) == j : v >= lo && v < hi && (v - lo) % 256 == tid) {
            mine = j;
            xy = to_f(row.x[j]);
        }
    }
    const f2 nref = pk(-st.m, -st.m), cc = pk(c2, c2), k2 = pk(kq, kq);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lo + i * 256 + tid;
        if (v < hi) {
            f2 f[N / 2];
            Vec<T>::wide(raw[i], f);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) f[j] = mul2(ex2x2(mul2(add2(f[j], nref), cc)), k2);
            store_vec<T>(dx + row.head + int64_t(v) * N, Vec<T>::narrow(f), whole);
        }
    }
    if (edge) dx[row.edge_at(tid)] = from_f<T>(ex2((xe - st.m) * c2) * kq);
    if (mine >= 0) dx[mine] = from_f<T>(__fmaf_rn(ex2((xy - st.m) * c2), kq, st.w));
}

// How a launch lays its rows out.
struct RowShape {
    int threads, nv, cluster;
};

template <typename T>
RowShape shape_for(int op, int64_t rows, int vocab, int sms) {
    const int vecs = (vocab + Vec<T>::N - 1) / Vec<T>::N;
    RowShape s{64, 4, 1};
    while (s.threads < 512 && s.threads * 4 < vecs) s.threads *= 2;
    if (s.threads * 4 < vecs) s.nv = 8;
    while (s.cluster < kMaxCluster && s.threads * s.nv * s.cluster < vecs) s.cluster *= 2;
    // few rows: spread each over more CTAs while the GPU has idle SMs and a thread more than one vector
    while (s.cluster < kMaxCluster && rows * s.cluster * 2 <= sms && s.threads * s.cluster < vecs) s.cluster *= 2;
    const int per = (vecs + s.cluster * s.threads - 1) / (s.cluster * s.threads);
    s.nv = per <= 2 ? 2 : per <= 4 ? 4 : 8;
    return s;
}

template <typename T, int OP, int NV, bool DUAL>
cudaError_t row_launch(const LossArgs& a, const RowShape& sh, int sms, cudaStream_t s) {
    auto* kernel = k_row<T, OP, NV, DUAL>;
    const size_t smem = OP == kDistill ? sizeof(float) * 2 * 3 * size_t(a.k + 1) : 0;
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, sh.threads, smem);
    if (e != cudaSuccess) return e;
    int64_t groups = int64_t(per_sm) * sms / sh.cluster;
    if (groups > kMaxLossClusters) groups = kMaxLossClusters;
    if (groups > a.rows) groups = a.rows;
    if (groups < 1) groups = 1;
    const int t = int(1.0f / a.it + 0.5f);
    const int pow = DUAL && t >= 2 && t <= 4 && a.it == 1.0f / float(t) ? t : 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(groups * sh.cluster));
    cfg.blockDim = dim3(unsigned(sh.threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(sh.cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = sh.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, int(sh.cluster), pow);
}

template <typename T, int OP, bool DUAL>
cudaError_t rows_by_nv(const LossArgs& a, const RowShape& sh, int sms, cudaStream_t s) {
    if (sh.nv == 2) return row_launch<T, OP, 2, DUAL>(a, sh, sms, s);
    if (sh.nv == 4) return row_launch<T, OP, 4, DUAL>(a, sh, sms, s);
    return row_launch<T, OP, 8, DUAL>(a, sh, sms, s);
}

template <typename T>
cudaError_t rows_by_op(int op, const LossArgs& a, int sms, cudaStream_t s) {
    const RowShape sh = shape_for<T>(op, a.rows, a.vocab, sms);
    switch (op) {
        case kLogprob: return rows_by_nv<T, kLogprob, false>(a, sh, sms, s);
        case kPolicy: return rows_by_nv<T, kPolicy, false>(a, sh, sms, s);
        case kPrefStat: return rows_by_nv<T, kPrefStat, false>(a, sh, sms, s);
        default: break;
    }
    if (a.k > 0 && a.ce_weight > 0.0f && a.it != 1.0f) return rows_by_nv<T, kDistill, true>(a, sh, sms, s);
    return rows_by_nv<T, kDistill, false>(a, sh, sms, s);
}

template <typename T>
cudaError_t pref_grad(const LossArgs& a, cudaStream_t s) {
    const int vecs = (a.vocab + Vec<T>::N - 1) / Vec<T>::N;
    constexpr int NV = 4;
    const int64_t segs = vecs <= NV * 256 ? 1 : (vecs + NV * 256 - 1) / (NV * 256);
    if (a.rows * segs > 0x7fffffff) return cudaErrorInvalidValue;
    k_pref_grad<T, NV><<<unsigned(a.rows * segs), 256, 0, s>>>(a, int(segs));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_loss_rows(int op, int dt, const LossArgs& a, int sm_count, cudaStream_t s) {
    if (dt == kF32) return rows_by_op<float>(op, a, sm_count, s);
    if (dt == kBF16) return rows_by_op<__nv_bfloat16>(op, a, sm_count, s);
    return rows_by_op<__half>(op, a, sm_count, s);
}

cudaError_t launch_pref_grad(int dt, const LossArgs& a, cudaStream_t s) {
    if (dt == kF32) return pref_grad<float>(a, s);
    if (dt == kBF16) return pref_grad<__nv_bfloat16>(a, s);
    return pref_grad<__half>(a, s);
}

}  // namespace tl
