// tl_stats_kernels.cu - softmax statistics of vocabulary logits, their largest entries, and the
// gradient of log-probabilities and entropies (tl_token_stats, tl_token_grad of include/tl_loss.h).
//
// Mathematics.  For one row x of V logits, it = 1 / temperature, c2 = it log2 e, M = max x, and
// w_j = x_j c2 - u with the whole number u next to M c2 (or w_j = (x_j - M) c2, see big()):
//   S = sum_j 2^w_j,  W = sum_j w_j 2^w_j,  log q_j = ln 2 (w_j - log2 S),
//   H = -sum_j q_j log q_j = ln 2 (log2 S - W / S).
// So one pass with one exponential, two sums and a maximum gives log-probabilities and entropy, and
// sums against other u join by exact powers of two: 2^d S and 2^d (W + d S).
#include "tl_loss_device.cuh"

namespace tl {
namespace {

// ---------------------------------------------------------------------------
// Sums of a part of a row
// ---------------------------------------------------------------------------

// From exponents against a part's reference m to those against `to`: what is added.
__device__ __forceinline__ float exponent_step(float m, float to, float c2) {
    if (!big(to, c2)) return big(m, c2) ? __fmaf_rn(m, c2, -anchor(to, c2)) : anchor(m, c2) - anchor(to, c2);
    return (m - to) * c2 - (big(m, c2) ? 0.0f : __fmaf_rn(m, c2, -anchor(m, c2)));
}
// S and W of a part with reference m, against `to`.  An empty part's 0 (or NaN) stays.
__device__ __forceinline__ void move_sums(float m, float to, float c2, float& s, float& w) {
    if (m == kNegInf || m == to) return;
    const float d = exponent_step(m, to, c2);
    const float f = !big(to, c2) && !big(m, c2) ? power_of_two(fminf(d, 127.0f)) : ex2(d);
    w = f != 0.0f ? f * __fmaf_rn(d, s, w) : 0.0f;
    s *= f;
}

// An exponent far below every other: 2^kLowest is 0, and 0 times it as well (an excluded entry's
// own exponent is -inf, and 0 times that is not).
constexpr float kLowest = -200.0f;

// The exponent of x against the reference m.
__device__ __forceinline__ float exponent(float x, float m, float c2) {
    return fmaxf(big(m, c2) ? (x - m) * c2 : __fmaf_rn(x, c2, -anchor(m, c2)), kLowest);
}

// log q of an entry x of a row with a softmax.  Roundings of the sum are not let above 0, and an entry at
// a type's lowest value, whose exponent overflows, has its distance.
__device__ __forceinline__ float log_q(float x, float M, float u, float c2, bool far, float S, float it) {
    const float r = log_share(x, M, u, c2, far, S);
    return fminf(r == kNegInf ? (x - M) * it : r, 0.0f);
}

// ---------------------------------------------------------------------------
// The largest entries
// ---------------------------------------------------------------------------

// Order of logits as whole numbers (-0 like 0), and back.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t order) {
    return __uint_as_float(order & 0x80000000u ? order & 0x7fffffffu : ~order);
}
constexpr uint32_t kLeast = 0x00800000u;   // the least order above that of -inf

// A candidate: the larger one comes first (higher logit, then lower id).
__device__ __forceinline__ unsigned long long candidate(uint32_t order, int id) {
    return (static_cast<unsigned long long>(order) << 32) | uint32_t(~id);
}

constexpr int kGroupsPerThread = 8;
constexpr int kCandidates = 1024;

// The sum of v over the CTA; `sh` holds 2 x B / 32 numbers, used in turns (`turn` flips).
template <int B> __device__ __forceinline__ int cta_sum(int v, int (*sh)[B / 32], int& turn) {
    const int warp = threadIdx.x >> 5;
    v = __reduce_add_sync(~0u, v);
    if ((threadIdx.x & 31) == 0) sh[turn][warp] = v;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int i = 0; i < B / 32; ++i) all += sh[turn][i];
    turn ^= 1;
    return all;
}

// ---------------------------------------------------------------------------
// A CTA per row
// ---------------------------------------------------------------------------

// The largest k entries without a second pass over the row.  The row's vectors fall into groups (a
// thread's consecutive ones, at most eight groups per thread) whose maxima the softmax's pass gives for
// nothing.  Let t be the k-th largest of these maxima: k groups have an entry >= t each, so every
// one of the k largest entries is >= t, and lies in a group whose maximum is.  Those groups (k, and a
// few that the search for t leaves) are read again, out of L2, their entries >= t are the
// candidates, and a candidate's place is the number of candidates before it.
//
// Where more candidates come together than fit (thousands of equal entries, or the largest ones
// side by side in a few groups), the exact k-th entry is searched for in the row itself: every count
// is a pass out of L2.
template <typename T, int B>
__global__ void __launch_bounds__(B) k_stats(const StatsArgs a) {
    constexpr int N = Vec<T>::N, nw = B / 32, G = kGroupsPerThread;
    __shared__ float4 parts[nw];
    extern __shared__ unsigned long long found[];                  // kCandidates
    float(*const gmax)[B] = reinterpret_cast<float(*)[B]>(found + kCandidates);   // [G][B]
    __shared__ int sums[2][nw], nfound;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float c2 = a.it * kLog2e, kNaN = __int_as_float(0x7fffffff);
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t y = a.target ? a.target[r] : 0;
        auto put = [&](int i, int id, float lp) {
            const int64_t at = r * a.ld_top + i;
            if (a.id_bytes == 8) static_cast<int64_t*>(a.top_id)[at] = id; else static_cast<int32_t*>(a.top_id)[at] = id;
            a.top_logp[at] = lp;
        };
        if (y < 0) {
            for (int i = tid; i < a.k; i += B) put(i, -1, 0.0f);
            if (tid == 0) {
                if (a.logp) a.logp[r] = 0.0f;
                if (a.entropy) a.entropy[r] = 0.0f;
                if (a.saved) for (int i = 0; i < 3; ++i) a.saved[3 * r + i] = 0.0f;
            }
            continue;
        }
        const T* const x = static_cast<const T*>(a.x) + r * a.ld;
        const Place<T> pl(x, a.vocab, 0, 0);
        const T* const body = x + pl.head;
        const bool edge = tid < pl.edges;
        const float xe = edge ? to_f(x[pl.edge_at(tid)]) : kNegInf;
        const int per = (pl.body + B - 1) / B, size = (per + G - 1) / G;   // vectors per thread, per group
        // one pass: the largest entry, and the sums against a reference near it
        float top = kNegInf, m = kNegInf, s = 0.0f, w = 0.0f;
        for (int g = 0; g < G; ++g) {
            float gm = kNegInf;
            for (int i = g * size; i < min(per, (g + 1) * size); ++i) {
                const int v = tid + B * i;
                if (v >= pl.body) break;
                float f[N];
                const uint4 raw = ld16(body + int64_t(v) * N);
                const float vt = Vec<T>::top(raw);
                gm = fmaxf(gm, vt);
                if (vt > m) {
                    move_sums(m, vt, c2, s, w);
                    m = vt;
                }
                Vec<T>::wide(raw, f);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (f[j] != f[j]) s = kNaN;
                    const float z = exponent(f[j], part_ref(m), c2), e = ex2(z);
                    s += e;
                    w = __fmaf_rn(e, z, w);
                }
            }
            if (a.k > 0) gmax[g][tid] = gm;
            top = fmaxf(top, gm);
        }
        if (xe != xe) s = kNaN;
        // the warp's part, edges included, then the CTA's
        const float wt = warp_max(fmaxf(top, xe)), ref = part_ref(wt);
        move_sums(m, ref, c2, s, w);
        if (edge && xe == xe) {
            const float z = exponent(xe, ref, c2), e = ex2(z);
            s += e;
            w = __fmaf_rn(e, z, w);
        }
        s = warp_sum(s);
        w = warp_sum(w);
        __syncthreads();
        if (lane == 0) parts[warp] = make_float4(wt, s, w, 0.0f);
        if (tid == 0) nfound = 0;
        __syncthreads();
        const float4 p = lane < nw ? parts[lane] : make_float4(kNegInf, 0.0f, 0.0f, 0.0f);
        const float M = warp_max(p.x);
        s = p.y;
        w = p.z;
        move_sums(p.x, part_ref(M), c2, s, w);
        const float S = warp_sum(s), W = warp_sum(w);
        const bool none = !(fabsf(M) < INFINITY) || S != S;   // no softmax
        const bool far = big(M, c2);
        const float u = anchor(M, c2);
        auto share = [&](float x) { return none ? kNaN : log_q(x, M, u, c2, far, S, a.it); };
        if (tid == 0) {
            const float log_sum = -share(M);
            const float H = fmaxf(log_sum + ((far ? 0.0f : __fmaf_rn(M, c2, -u)) - W / S) * kLn2, 0.0f);
            if (a.logp) a.logp[r] = y < a.vocab ? share(to_f(x[y])) : kNaN;
            if (a.entropy) a.entropy[r] = none ? kNaN : H;
            if (a.saved) {
                a.saved[3 * r] = none ? kNaN : M;
                a.saved[3 * r + 1] = log_sum;
                a.saved[3 * r + 2] = none ? kNaN : H;
            }
        }
        if (a.k == 0) continue;
        if (none) {
            for (int i = tid; i < a.k; i += B) put(i, -1, kNaN);
            continue;
        }
        // t: at least k groups are >= lo, fewer than k are >= hi
        uint32_t key[G];
#pragma unroll
        for (int g = 0; g < G; ++g) key[g] = order_of(gmax[g][tid]);
        auto groups_from = [&](uint32_t t) {
            int n = 0;
#pragma unroll
            for (int g = 0; g < G; ++g) n += key[g] >= t;
            return cta_sum<B>(n, sums, turn);
        };
        uint32_t lo = kLeast, hi = order_of(M) + 1;
        int over = groups_from(lo);
        while (over > a.k + a.k / 2 + 16 && hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            const int n = groups_from(mid);
            if (n >= a.k) { lo = mid; over = n; } else { hi = mid; }
        }
        auto offer = [&](float v, int id) {
            const uint32_t o = order_of(v);
            if (o < lo) return;
            const int i = atomicAdd(&nfound, 1);
            if (i < kCandidates) found[i] = candidate(o, id);
        };
        for (int g = 0; g < G; ++g) {
            if (key[g] < lo) continue;
            for (int i = g * size; i < min(per, (g + 1) * size); ++i) {
                const int v = tid + B * i;
                if (v >= pl.body) break;
                float f[N];
                Vec<T>::wide(ld16(body + int64_t(v) * N), f);
#pragma unroll
                for (int j = 0; j < N; ++j) offer(f[j], pl.head + v * N + j);
            }
        }
        if (edge) offer(xe, pl.edge_at(tid));
        __syncthreads();
        if (nfound > kCandidates) {
            // the k-th largest entry itself: at least k entries are >= lo, fewer than k are >= hi
            auto entries_from = [&](uint32_t t) {
                int n = 0;
                for (int j = tid; j < a.vocab; j += B) n += order_of(to_f(x[j])) >= t;
                return cta_sum<B>(n, sums, turn);
            };
            hi = order_of(M) + 1;
            bool first = true;   // thousands of equal entries: the next order already has fewer than k
            while (hi - lo > 1) {
                const uint32_t mid = first ? lo + 1 : lo + (hi - lo) / 2;
                first = false;
                if (entries_from(mid) >= a.k) lo = mid; else hi = mid;
            }
            __syncthreads();
            if (tid == 0) nfound = 0;
            __syncthreads();
            for (int j = tid; j < a.vocab; j += B) {   // fewer than k
                const uint32_t o = order_of(to_f(x[j]));
                if (o > lo) found[atomicAdd(&nfound, 1)] = candidate(o, j);
            }
            __syncthreads();
            int have = nfound;
            __syncthreads();
            // of those equal to the k-th the first ones
            for (int base = 0; have < a.k && base < a.vocab; base += B) {
                const int j = base + tid;
                const bool equal = j < a.vocab && order_of(to_f(x[j])) == lo;
                const unsigned ones = __ballot_sync(~0u, equal);
                if (lane == 0) sums[turn][warp] = __popc(ones);
                __syncthreads();
                int before = __popc(ones & ((1u << lane) - 1)), all = 0;
#pragma unroll
                for (int i = 0; i < nw; ++i) {
                    before += i < warp ? sums[turn][i] : 0;
                    all += sums[turn][i];
                }
                turn ^= 1;
                if (equal && have + before < a.k) found[have + before] = candidate(lo, j);
                have += all;
            }
            if (tid == 0) nfound = min(have, a.k);
            __syncthreads();
        }
        const int n = nfound;
        for (int i = tid; i < n; i += B) {
            const unsigned long long c = found[i];
            int place = 0;
            for (int j = 0; j < n; ++j) place += found[j] > c;
            if (place < a.k) put(place, int(~uint32_t(c)), share(logit_of(uint32_t(c >> 32))));
        }
        for (int i = n + tid; i < a.k; i += B) put(i, -1, kNegInf);
        __syncthreads();   // the next row writes the counters again
    }
}

template <typename T>
cudaError_t stats(const StatsArgs& a, int sms, GroupCache& cache, cudaStream_t s) {
    constexpr int B = 256;
    auto* kernel = k_stats<T, B>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(B);
    cfg.dynamicSmemBytes = kCandidates * 8 + kGroupsPerThread * B * 4;
    cfg.stream = s;
    int groups = 0;
    cudaError_t e = resident_groups(reinterpret_cast<const void*>(kernel), cfg, RowShape{B, 0}, sms, cache, groups);
    if (e != cudaSuccess) return e;
    cfg.gridDim.x = unsigned(groups < a.rows ? groups : a.rows);
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// ---------------------------------------------------------------------------
// The gradient
// ---------------------------------------------------------------------------

// With q_j = 2^(w_j - rest) of the saved statistics,
//   dx_j = -step q_j (ga + gb (log q_j + H)) + [j = y] step ga = 2^w_j (A + B w_j) + [j = y] step ga:
// one exponential and four multiplications or additions per element, every element on its own.  One
// segment of a row per CTA.
template <typename T, int NV, int TB>
__global__ void __launch_bounds__(TB) k_token_grad(const TokenGradArgs a, const int segs) {
    constexpr int N = Vec<T>::N;
    const int tid = threadIdx.x;
    const int64_t r = int64_t(blockIdx.x) / segs;
    const int seg = int(int64_t(blockIdx.x) - r * segs);
    const T* const x = static_cast<const T*>(a.x) + r * a.ld;
    const Place<T> row(x, a.vocab, 0, 0);
    T* const dx = static_cast<T*>(a.dx) + r * a.ldd;
    const bool whole = same_phase(x, static_cast<const T*>(dx));
    const T* const body = x + row.head;
    // segments end on 128-byte boundaries: the first one is short by `off` vectors
    const int lo = seg * NV * TB - row.off, hi = min(row.body, lo + NV * TB);
    const bool edge = seg == 0 && tid < row.edges;
    const int64_t y = a.target ? a.target[r] : 0;
    if (y < 0) {
        for (int v = lo + tid; v < hi; v += TB)
            if (v >= 0) store_vec<T>(dx + row.head + int64_t(v) * N, make_uint4(0, 0, 0, 0), whole);
        if (edge) dx[row.edge_at(tid)] = from_f<T>(0.0f);
        return;
    }
    uint4 raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lo + i * TB + tid;
        if (v >= 0 && v < hi) raw[i] = ld16(body + int64_t(v) * N);
    }
    const float xe = edge ? to_f(x[row.edge_at(tid)]) : 0.0f;
    const float c2 = a.it * kLog2e, kNaN = __int_as_float(0x7fffffff);
    const float M = a.saved[3 * r], H = a.saved[3 * r + 2];
    const bool far = big(M, c2);
    const float u = far ? 0.0f : anchor(M, c2), base = far ? M : 0.0f;
    // log2 q_j = w_j - rest
    const float rest = __fmaf_rn(a.saved[3 * r + 1], kLog2e, far ? 0.0f : __fmaf_rn(M, c2, -u));
    const float step = (a.seed ? *a.seed : 1.0f) * a.it;
    const float ga = a.grad_logp ? a.grad_logp[r] : 0.0f, gb = a.grad_entropy ? a.grad_entropy[r] : 0.0f;
    const float scale = -step * ex2(-rest) + (y >= a.vocab ? kNaN : 0.0f);
    const float A = scale * __fmaf_rn(gb, __fmaf_rn(-rest, kLn2, H), ga), B = scale * gb * kLn2, at_label = step * ga;
    auto value = [&](float v) {
        const float w = fmaxf(__fmaf_rn(v - base, c2, -u), kLowest);
        return ex2(w) * __fmaf_rn(w, B, A);
    };
    // the label's element: in vector yv, or at an edge
    const int yj = a.grad_logp && y < a.vocab ? int(y) : -1;
    const int yv = yj >= row.head ? (yj - row.head) / N : -1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lo + i * TB + tid;
        if (v >= 0 && v < hi) {
            float f[N];
            Vec<T>::wide(raw[i], f);
#pragma unroll
            for (int j = 0; j < N; ++j) f[j] = value(f[j]);
            if (v == yv) {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (row.head + v * N + j == yj) f[j] += at_label;
            }
            store_vec<T>(dx + row.head + int64_t(v) * N, Vec<T>::narrow(f), whole);
        }
    }
    if (edge) dx[row.edge_at(tid)] = from_f<T>(value(xe) + (row.edge_at(tid) == yj ? at_label : 0.0f));
}

template <typename T, int TB>
cudaError_t token_grad_by(const TokenGradArgs& a, cudaStream_t s) {
    constexpr int NV = 4;
    const int64_t vecs = (int64_t(a.vocab) + Vec<T>::N - 1) / Vec<T>::N, segs = (vecs + 7 + NV * TB - 1) / (NV * TB);
    if (a.rows * segs > 0x7fffffff) return cudaErrorInvalidValue;
    k_token_grad<T, NV, TB><<<unsigned(a.rows * segs), TB, 0, s>>>(a, int(segs));
    return cudaGetLastError();
}
template <typename T> cudaError_t token_grad(const TokenGradArgs& a, cudaStream_t s) {
    const int places = (a.vocab + Vec<T>::N - 1) / Vec<T>::N + 7;
    if (places <= 4 * 64) return token_grad_by<T, 64>(a, s);
    return places <= 4 * 128 ? token_grad_by<T, 128>(a, s) : token_grad_by<T, 256>(a, s);
}

}  // namespace

cudaError_t launch_token_stats(int dt, const StatsArgs& a, int sm_count, GroupCache& cache, cudaStream_t s) {
    if (dt == kF32) return stats<float>(a, sm_count, cache, s);
    if (dt == kBF16) return stats<__nv_bfloat16>(a, sm_count, cache, s);
    return stats<__half>(a, sm_count, cache, s);
}

cudaError_t launch_token_grad(int dt, const TokenGradArgs& a, cudaStream_t s) {
    if (dt == kF32) return token_grad<float>(a, s);
    if (dt == kBF16) return token_grad<__nv_bfloat16>(a, s);
    return token_grad<__half>(a, s);
}

}  // namespace tl
