// tl_loss_device.cuh - what the kernels over vocabulary logits share: exponentials against a
// reference, logarithms of shares, 16-byte vectors of a row at any alignment, barriers, asynchronous
// copies, and the number of row groups that fit the device.
#pragma once

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
// n, rest: log2_parts of s.
__device__ __forceinline__ float log_share(float x, float m, float u, float c, bool far, float n, float rest) {
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
__device__ __forceinline__ float log_share(float x, float m, float u, float c, bool far, float s) {
    float n, rest;
    log2_parts(s, n, rest);
    return log_share(x, m, u, c, far, n, rest);
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

// Named barriers: `count` threads take part; arrive does not wait.
__device__ __forceinline__ void bar_sync(int id, int count) {
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int count) {
    __syncwarp();
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
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

__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

constexpr int kMaxRingBytes = 220 * 1024;   // dynamic shared memory: tiles and teacher entries

// How a launch lays its rows out: threads per CTA, and CTAs per row (2^clog).
struct RowShape {
    int threads, clog;
};

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

}  // namespace
}  // namespace tl
