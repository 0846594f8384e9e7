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

// (x - m) / 2: it is in fp32 where x - m is not (a type's largest and lowest value in one row), and halving
// rounds nothing above 2^-126.  Doubled scales are in fp32 too (temperatures are normal numbers).
__device__ __forceinline__ float half_apart(float x, float m) { return __fmaf_rn(0.5f, x, -0.5f * m); }
// (x - m) c.
__device__ __forceinline__ float distance(float x, float m, float c) { return half_apart(x, m) * (2.0f * c); }

// From exponents against a part's reference m to those against `to`: what is added.
__device__ __forceinline__ float exponent_step(float m, float to, float c2) {
    if (!big(to, c2)) return big(m, c2) ? __fmaf_rn(m, c2, -anchor(to, c2)) : anchor(m, c2) - anchor(to, c2);
    return distance(m, to, c2) - (big(m, c2) ? 0.0f : __fmaf_rn(m, c2, -anchor(m, c2)));
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

// ---------------------------------------------------------------------------
// Pairs of fp32 in one register pair: two multiply-adds or additions to an instruction
// ---------------------------------------------------------------------------

typedef unsigned long long pair_t;
__device__ __forceinline__ pair_t pair_of(float a, float b) {
    pair_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void apart(pair_t p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ pair_t fma_pair(pair_t a, pair_t b, pair_t c) {
    pair_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ pair_t add_pair(pair_t a, pair_t b) {
    pair_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// The larger, the smaller of both, NaN if v is.
__device__ __forceinline__ float max_nan(float v, float least) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(least));
    return r;
}
__device__ __forceinline__ float min_nan(float v, float most) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(most));
    return r;
}

// log2(e) / temperature, and what its rounding left out: with fp32 logits it is counted too, where an entropy
// shows it (temperature 0.72, whose scale rounds by 5e-8: off by 1.2e-7 of itself without, 7e-8 with it); 16-bit ones
// have no time for it.
struct Scale {
    float c2, low;
    __device__ __forceinline__ Scale(const StatsArgs& a) : c2(a.c2), low(a.c2_low) {}
};

// 2^z for |z| <= 1/2 or a little above: the series of e^(z ln 2), whose ninth term is below 2^-27.
__device__ __forceinline__ float power_near_1(float z) {
    const float t = z * kLn2;
    float p = 1.0f / 5040.0f;
    p = __fmaf_rn(p, t, 1.0f / 720.0f);
    p = __fmaf_rn(p, t, 1.0f / 120.0f);
    p = __fmaf_rn(p, t, 1.0f / 24.0f);
    p = __fmaf_rn(p, t, 1.0f / 6.0f);
    p = __fmaf_rn(p, t, 0.5f);
    p = __fmaf_rn(p, t, 1.0f);
    return __fmaf_rn(p, t, 1.0f);
}

// A thread's sums over the elements that it has seen, against a reference near its largest one.
template <typename T> struct Running {
    static constexpr int N = Vec<T>::N, U = 4;
    float m = kNegInf, limit = kNegInf, s = 0.0f, w = 0.0f;
    float s_left = 0.0f, w_left = 0.0f;   // fp32 logits: what the sums' additions left out; 16-bit ones have no time for it
    float u = 0.0f;      // the reference's whole number
    bool slow = false;   // element by element, see below

    // Vectors with an excluded entry (-inf) are summed again, their logits held above this one (16-bit ones before
    // they are widened; 32-bit ones' exponents are held as well).  That needs it to be far below the reference, 2^-150
    // of it, which very large temperatures do not leave, and its exponent to be in fp32, which very small ones do not.
    static constexpr float kFloor = sizeof(T) == 4 ? -3.4e38f : Vec<T>::kEmpty == 0xfc00fc00u ? -65504.0f : -9.9e29f;

    // To a much larger element.  Smaller steps are left: exponentials up to 2^32 of the reference do no harm.
    __device__ __forceinline__ void raise(float top, float c2) {
        if (!(top > limit)) return;
        fold();
        move_sums(m, top, c2, s, w);
        m = top;
        limit = m + 32.0f / c2;
        slow = big(m, c2) || !((m - kFloor) * c2 > 150.0f) || (sizeof(T) == 2 && !(kFloor * c2 > -3.4e38f));
        u = slow ? 0.0f : anchor(m, c2);
    }
    __device__ __forceinline__ void add_one(float v, const Scale& c) {
        const float ref = part_ref(m);
        const bool far = big(ref, c.c2);
        float z = far ? distance(v, ref, c.c2) : __fmaf_rn(v, c.c2, -anchor(ref, c.c2));
        if (sizeof(T) == 4 && v > kNegInf) z = far ? __fmaf_rn(half_apart(v, ref), 2.0f * c.low, z) : __fmaf_rn(v, c.low, z);
        z = max_nan(z, kLowest);
        const float e = ex2(z);
        s += e;
        w = __fmaf_rn(e, z, w);
    }
    // The sums of U vectors; HOLD: with elements held above kFloor.
    template <bool HOLD> __device__ __forceinline__ void sums_of(const uint4 (&raw)[U], const Scale& c, float& s_, float& w_) const {
        const pair_t uu = pair_of(-u, -u), c2c2 = pair_of(c.c2, c.c2), lolo = pair_of(c.low, c.low);
        pair_t s2 = 0, w2 = 0;   // of these vectors first: see tree_sum
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float f[N];
            Vec<T>::wide(HOLD ? held(raw[i]) : raw[i], f);
            if (HOLD && sizeof(T) == 4) {   // -inf times a negative low part
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] = max_nan(f[j], kFloor);
            }
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                pair_t z = fma_pair(pair_of(f[j], f[j + 1]), c2c2, uu);
                if (sizeof(T) == 4) z = fma_pair(pair_of(f[j], f[j + 1]), lolo, z);
                float z0, z1;
                apart(z, z0, z1);
                if (HOLD && sizeof(T) == 4) {
                    z0 = max_nan(z0, kLowest);
                    z1 = max_nan(z1, kLowest);
                    z = pair_of(z0, z1);
                }
                const pair_t e = pair_of(ex2(z0), ex2(z1));
                s2 = add_pair(s2, e);
                w2 = fma_pair(e, z, w2);
            }
        }
        float p0, p1;
        apart(s2, p0, p1);
        s_ = p0 + p1;
        apart(w2, p0, p1);
        w_ = p0 + p1;
    }
    // The sums of vectors with excluded or no entries, or (slow) element by element.
    __device__ __forceinline__ float2 held_sums(uint4 a, uint4 b, uint4 c, uint4 d, bool element_wise, const Scale& scale) const {
        Running<T> r;
        r.m = m;
        r.u = u;
        if (!element_wise) {
            const uint4 raw[U] = {a, b, c, d};
            r.template sums_of<true>(raw, scale, r.s, r.w);
        } else {
#pragma unroll 1
            for (int i = 0; i < U; ++i) {
                const uint4 v = i == 0 ? a : i == 1 ? b : i == 2 ? c : d;
                float f[N];
                Vec<T>::wide(v, f);
#pragma unroll
                for (int j = 0; j < N; ++j) r.add_one(f[j], scale);
            }
        }
        return make_float2(r.s, r.w);
    }
    // Out of line, where most batches do without (4,096 x 128,256 with 64 alternatives: 202 us, 206 in line; where
    // every batch is of this kind it is in line: 16,384 x 1,000 with 8 34 us, 38 out of line).
    static __device__ __noinline__ float2 held_sums_apart(uint4 a, uint4 b, uint4 c, uint4 d, bool element_wise, float m, float u, Scale scale) {
        Running<T> r;
        r.m = m;
        r.u = u;
        return r.held_sums(a, b, c, d, element_wise, scale);
    }
    // U vectors, of which the largest element has been through raise().  STREAM: whole: none of them is empty.
    template <bool STREAM> __device__ __forceinline__ void add(const uint4 (&raw)[U], bool whole, const Scale& c) {
        const bool element_wise = slow || m == kNegInf;
        float ds = 0.0f, dw = __int_as_float(0x7fffffff), left;
        if (STREAM && whole && !slow) sums_of<false>(raw, c, ds, dw);
        if (dw != dw) {   // 0 times an excluded entry's exponent, or a NaN entry
            const float2 d = STREAM ? held_sums_apart(raw[0], raw[1], raw[2], raw[3], element_wise, m, u, c)
                                    : held_sums(raw[0], raw[1], raw[2], raw[3], element_wise, c);
            ds = d.x;
            dw = d.y;
        }
        if (sizeof(T) == 4) {
            s = sum_parts(s, ds, left);
            s_left += left;
            w = sum_parts(w, dw, left);
            w_left += left;
        } else {
            s += ds;
            w += dw;
        }
    }
    __device__ __forceinline__ void fold() {
        if (sizeof(T) != 4) return;
        s += s_left;
        w += w_left;
        s_left = w_left = 0.0f;
    }
    // The exponential of the thread's largest element again, from its exponent in full and without the
    // hardware unit's error: the reference may be 32 bits below it, where the exponent rounds to 2^-20, and a row
    // that it dominates has nothing to average either error with (entropies off by 1.6e-7 of themselves where
    // labels have most of the probability, 5e-8 so).
    __device__ __forceinline__ void retake(float top, const Scale& c) {
        fold();
        if (slow || !(m > kNegInf) || !(__fmaf_rn(top, c.c2, -u) > -64.0f)) return;   // nothing, or too little to count
        const float low = sizeof(T) == 4 ? c.low : 0.0f;
        const float p = __fmul_rn(top, c.c2), pe = __fmaf_rn(top, low, __fmaf_rn(top, c.c2, -p));
        float left;
        const float at = sum_parts(p, -u, left), n = rintf(at), rest = left + pe;
        const float e = power_near_1((at - n) + rest) * __int_as_float((int(n) + 127) << 23);
        float z = __fmaf_rn(top, c.c2, -u);
        if (sizeof(T) == 4) z = __fmaf_rn(top, low, z);
        const float d = e - ex2(z);
        s += d;
        w += __fmaf_rn(e, (at - z) + rest, d * z);
    }
    static __device__ __forceinline__ uint4 held(uint4 v) {
        if constexpr (sizeof(T) == 2) {
            v.x = held2(v.x); v.y = held2(v.y); v.z = held2(v.z); v.w = held2(v.w);
        }
        return v;
    }
    static __device__ __forceinline__ uint32_t held2(uint32_t v) {
        uint32_t r = v;
        if constexpr (Vec<T>::kEmpty == 0xfc00fc00u)
            asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0xfbfffbffu));
        else
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0xf149f149u));
        return r;
    }
};

// The largest element of four vectors.
template <typename T> __device__ __forceinline__ float top_of(const uint4 (&raw)[4]) {
    return fmaxf(fmaxf(Vec<T>::top(raw[0]), Vec<T>::top(raw[1])), fmaxf(Vec<T>::top(raw[2]), Vec<T>::top(raw[3])));
}
template <> __device__ __forceinline__ float top_of<__nv_bfloat16>(const uint4 (&raw)[4]) {
    using V = Vec<__nv_bfloat16>;
    uint4 m = raw[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        const __nv_bfloat162 x = __hmax2(V::b2(m.x), V::b2(raw[i].x)), y = __hmax2(V::b2(m.y), V::b2(raw[i].y));
        const __nv_bfloat162 z = __hmax2(V::b2(m.z), V::b2(raw[i].z)), w = __hmax2(V::b2(m.w), V::b2(raw[i].w));
        m = make_uint4(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y),
                       *reinterpret_cast<const uint32_t*>(&z), *reinterpret_cast<const uint32_t*>(&w));
    }
    return V::top(m);
}
template <> __device__ __forceinline__ float top_of<__half>(const uint4 (&raw)[4]) {
    using V = Vec<__half>;
    uint4 m = raw[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        const __half2 x = __hmax2(V::h2(m.x), V::h2(raw[i].x)), y = __hmax2(V::h2(m.y), V::h2(raw[i].y));
        const __half2 z = __hmax2(V::h2(m.z), V::h2(raw[i].z)), w = __hmax2(V::h2(m.w), V::h2(raw[i].w));
        m = make_uint4(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y),
                       *reinterpret_cast<const uint32_t*>(&z), *reinterpret_cast<const uint32_t*>(&w));
    }
    return V::top(m);
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
// The digits of an order that differ among logits of the type.
template <typename T> struct Order;
template <> struct Order<float> { static constexpr int kShift = 0; };
template <> struct Order<__nv_bfloat16> { static constexpr int kShift = 16; };
template <> struct Order<__half> { static constexpr int kShift = 13; };
template <typename T> __device__ __forceinline__ uint32_t rank_of(float x) { return order_of(x) >> Order<T>::kShift; }
// The least rank above that of -inf.
template <typename T> constexpr uint32_t kLeast = 0x00800000u >> Order<T>::kShift;

// A candidate: the larger one comes first (higher logit, then lower id).
__device__ __forceinline__ unsigned long long candidate(uint32_t order, int id) {
    return (static_cast<unsigned long long>(order) << 32) | uint32_t(~id);
}

constexpr int kCandidates = 1024;

// Barrier `bar` of the SB threads that choose a row's entries.
template <int SB> __device__ __forceinline__ void sync(int bar) {
    if constexpr (SB == 32) __syncwarp(); else bar_sync(bar, SB);
}
// The sum of v over them; `sh` holds 2 x 8 numbers, used in turns (`turn` flips).
template <int SB> __device__ __forceinline__ int sum_over(int v, int (*sh)[8], int& turn, int tid, int bar) {
    v = __reduce_add_sync(~0u, v);
    if constexpr (SB == 32) return v;
    if ((tid & 31) == 0) sh[turn][tid >> 5] = v;
    sync<SB>(bar);
    v = 0;
#pragma unroll
    for (int i = 0; i < SB / 32; ++i) v += sh[turn][i];
    turn ^= 1;
    return v;
}

// More candidates than fit: the k-th largest entry itself.  At least k entries are >= lo, M is the
// largest.  Every count is a pass over the row, out of L2.  Gives the number of candidates, at most k.
template <typename T, int SB>
__device__ __noinline__ int exact_candidates(const T* x, int vocab, int k, uint32_t lo, float M, unsigned long long* found,
                                             int* nfound, int (*sh)[8], int turn, int tid, int bar) {
    const int warp = tid >> 5, lane = tid & 31;
    uint32_t hi = rank_of<T>(M) + 1;   // fewer than k are >= hi
    bool first = true;                 // thousands of equal entries: the next rank already has fewer than k
    while (hi - lo > 1) {
        const uint32_t mid = first ? lo + 1 : lo + (hi - lo) / 2;
        first = false;
        int c = 0;
        for (int j = tid; j < vocab; j += SB) c += rank_of<T>(to_f(x[j])) >= mid;
        if (sum_over<SB>(c, sh, turn, tid, bar) >= k) lo = mid; else hi = mid;
    }
    sync<SB>(bar);
    if (tid == 0) *nfound = 0;
    sync<SB>(bar);
    for (int j = tid; j < vocab; j += SB) {   // fewer than k
        const uint32_t o = order_of(to_f(x[j]));
        if (o >> Order<T>::kShift > lo) found[atomicAdd(nfound, 1)] = candidate(o, j);
    }
    sync<SB>(bar);
    int n = *nfound;
    // of those equal to the k-th the first ones
    for (int base = 0; n < k && base < vocab; base += SB) {
        const int j = base + tid;
        const uint32_t o = j < vocab ? order_of(to_f(x[j])) : 0u;
        const bool equal = j < vocab && o >> Order<T>::kShift == lo;
        const unsigned ones = __ballot_sync(~0u, equal);
        int before = __popc(ones & ((1u << lane) - 1)), all = __popc(ones);
        if constexpr (SB > 32) {
            if (lane == 0) sh[turn][warp] = all;
            sync<SB>(bar);
            all = 0;
#pragma unroll
            for (int v = 0; v < SB / 32; ++v) {
                before += v < warp ? sh[turn][v] : 0;
                all += sh[turn][v];
            }
            turn ^= 1;
        }
        if (equal && n + before < k) found[n + before] = candidate(o, j);
        n += all;
    }
    sync<SB>(bar);
    return min(n, k);
}

__device__ __forceinline__ int warp_before(int n, int& all) {   // the sum over the lanes below, and over all
    int to = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int below = __shfl_up_sync(~0u, to, o);
        if ((threadIdx.x & 31) >= o) to += below;
    }
    all = __shfl_sync(~0u, to, 31);
    return to - n;
}

// The n candidates in order, from the largest: settle(candidate, place) by one thread each.  They are
// dealt into 256 bins by rank, from M's down to lo's, the bins' starts are sums of counts, and within a bin
// (equal logits, or fp32 ones close by) a candidate's place is the number of larger ones.  `order` holds n
// numbers, `bins` 256.  (A bitonic network over 85 candidates took a warp 5,000 to 9,000 cycles beside
// busy ones, every pair counted as much.)
constexpr int kBins = 256;
// Up to so many are counted pair by pair: 16,384 x 1,000 bf16 with 8 alternatives (11 candidates) 29.8 us counted, 31.9 in bins,
// with 32 (40) 43.1 / 40.0; 4,096 x 8,192 with 8 31.4 / 34.8.
constexpr int kCounted = 24;
template <typename T, int SB, typename F>
__device__ __forceinline__ void place_candidates(const unsigned long long* found, int n, uint32_t lo, float M, int k, int* bins,
                                                 uint16_t* order, int tid, int bar, F settle) {
    if (n <= kCounted) {   // few: counted, without a barrier
        for (int i = tid; i < n; i += SB) {
            const unsigned long long c = found[i];
            int place = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) place += found[j] > c;
            if (place < k) settle(c, place);
        }
        return;
    }
    const uint32_t top = rank_of<T>(M), range = top - lo;
    const int shift = range < kBins ? 0 : 32 - 8 - __clz(range);
    auto bin_of = [&](unsigned long long c) { return (top - (uint32_t(c >> 32) >> Order<T>::kShift)) >> shift; };
    for (int i = tid; i < kBins; i += SB) bins[i] = 0;
    sync<SB>(bar);
    for (int i = tid; i < n; i += SB) atomicAdd(&bins[bin_of(found[i])], 1);
    sync<SB>(bar);
    if (tid < 32) {
        int4* const mine = reinterpret_cast<int4*>(bins) + 2 * tid;
        int4 p = mine[0], q = mine[1];
        int all;
        int at = warp_before(p.x + p.y + p.z + p.w + q.x + q.y + q.z + q.w, all);
        int next;
        next = at + p.x; p.x = at; at = next;
        next = at + p.y; p.y = at; at = next;
        next = at + p.z; p.z = at; at = next;
        next = at + p.w; p.w = at; at = next;
        next = at + q.x; q.x = at; at = next;
        next = at + q.y; q.y = at; at = next;
        next = at + q.z; q.z = at; at = next;
        q.w = at;
        mine[0] = p;
        mine[1] = q;
    }
    sync<SB>(bar);
    for (int i = tid; i < n; i += SB) order[atomicAdd(&bins[bin_of(found[i])], 1)] = uint16_t(i);
    sync<SB>(bar);   // now a bin's number is its end
    for (int i = tid; i < n; i += SB) {
        const unsigned long long c = found[i];
        const uint32_t bin = bin_of(c);
        int place = bin == 0 ? 0 : bins[bin - 1];
        if (place >= k) continue;
        const int end = bins[bin];
        for (int j = place; j < end; ++j) place += found[order[j]] > c;
        if (place < k) settle(c, place);
    }
}

// Other CTAs' shared memory.
__device__ __forceinline__ uint32_t remote_address(const void* smem, uint32_t rank) {
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(smem)), to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
    return to;
}
__device__ __forceinline__ void store_remote(uint32_t to, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(v) : "memory");
}
__device__ __forceinline__ int add_remote(uint32_t to, int v) {
    int r;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(to), "r"(v) : "memory");
    return r;
}

// What a row's sums amount to; by every lane of a warp, whose lanes 0 .. n - 1 (n <= PARTS) hold the parts
// (largest entry, S, W, and the least of the threads' largest entries).
struct RowSums {
    float M, S, W, least;
};
template <int PARTS> __device__ __forceinline__ RowSums join_parts(float4 p, float c2) {
    RowSums r;
    r.M = warp_max(p.x);
    r.least = -warp_max(-p.w);
    move_sums(p.x, part_ref(r.M), c2, p.y, p.z);
#pragma unroll
    for (int o = PARTS / 2; o > 0; o >>= 1) {
        p.y += __shfl_xor_sync(~0u, p.y, o);
        p.z += __shfl_xor_sync(~0u, p.z, o);
    }
    r.S = __shfl_sync(~0u, p.y, 0);
    r.W = __shfl_sync(~0u, p.z, 0);
    return r;
}
// The warp's part of them, its edge elements (-inf: none) included.
template <typename T> __device__ __forceinline__ float4 warp_part(Running<T>& t, float top, float xe, bool edge, const Scale& c) {
    t.retake(top, c);
    const float wt = warp_max(fmaxf(top, xe)), ref = part_ref(wt), least = -warp_max(-top);
    move_sums(t.m, ref, c.c2, t.s, t.w);
    t.m = ref;
    if (edge) t.add_one(xe, c);
    return make_float4(wt, warp_sum(t.s), warp_sum(t.w), least);
}

// A row's softmax, and its outputs.
struct RowSoftmax {
    float M, S, W, u, c2, low, it, n, rest;
    bool none, far;   // none: no softmax
    // fp32: whether the scale's low part counts (Scale)
    __device__ __forceinline__ RowSoftmax(const RowSums& r, const StatsArgs& a, bool fp32)
        : M(r.M), S(r.S), W(r.W), u(anchor(r.M, a.c2)), c2(a.c2), low(fp32 ? a.c2_low : 0.0f), it(a.it), none(!(fabsf(r.M) < INFINITY) || r.S != r.S),
          far(big(r.M, a.c2)) {
        log2_parts(S, n, rest);
    }
    // log q of an entry x.  Roundings of the sum are not let above 0, and an entry at a type's lowest value,
    // whose exponent overflows, has its distance (-inf where that is beyond fp32 as well).
    __device__ __forceinline__ float share(float x) const {
        if (none) return __int_as_float(0x7fffffff);
        if (x == kNegInf) return kNegInf;
        const float below = far ? __fmaf_rn(half_apart(M, x), 2.0f * low, rest) : __fmaf_rn(-x, low, rest);
        const float r = log_share(x, M, u, c2, far, n, fabsf(below) < INFINITY ? below : rest);
        return min_nan(r == kNegInf ? __fmaf_rn(-(n + rest), kLn2, distance(x, M, it)) : r, 0.0f);
    }
    // By a warp; xy: the label's logit.
    __device__ __forceinline__ void finish(const StatsArgs& a, int64_t r, int64_t y, float xy) const {
        const float kNaN = __int_as_float(0x7fffffff), log_sum = -share(M), lp = share(xy);
        const float H = max_nan(log_sum + ((far ? 0.0f : __fmaf_rn(M, low, __fmaf_rn(M, c2, -u))) - W / S) * kLn2, 0.0f);
        if ((threadIdx.x & 31) != 0) return;
        if (a.logp) a.logp[r] = y < a.vocab ? lp : kNaN;
        if (a.entropy) a.entropy[r] = none ? kNaN : H;
        if (a.saved) {
            a.saved[3 * r] = none ? kNaN : M;
            a.saved[3 * r + 1] = log_sum;
            a.saved[3 * r + 2] = none ? kNaN : H;
        }
    }
};
__device__ __forceinline__ void put_entry(const StatsArgs& a, int64_t r, int i, int id, float lp) {
    const int64_t at = r * a.ld_top + i;
    if (a.id_bytes == 8) static_cast<int64_t*>(a.top_id)[at] = id; else static_cast<int32_t*>(a.top_id)[at] = id;
    a.top_logp[at] = lp;
}
// An ignored row's outputs, by n threads.
__device__ __forceinline__ void ignored_row(const StatsArgs& a, int64_t r, int tid, int n) {
    for (int i = tid; i < a.k; i += n) put_entry(a, r, i, -1, 0.0f);
    if (tid == 0) {
        if (a.logp) a.logp[r] = 0.0f;
        if (a.entropy) a.entropy[r] = 0.0f;
    }
    if (tid < 3 && a.saved) a.saved[3 * r + tid] = 0.0f;
}

// ---------------------------------------------------------------------------
// Rows through shared memory
// ---------------------------------------------------------------------------

// The rows of a group, in tiles of TV vectors per thread, ST of them in shared memory, copied
// asynchronously ahead of their use in the order of it.  A thread copies the vectors that it will itself
// use, so a tile needs no barrier.
template <typename T, int B, int TV, int ST> struct Feed {
    static constexpr int N = Vec<T>::N, tile = B * TV;
    const StatsArgs& a;
    const int ngroups, rank, clog, tid;
    const bool alike;   // all rows lie alike where their stride is a multiple of 128 bytes
    const Place<T> first;
    int64_t fr, fynext;
    uint4* const ring;         // this thread's first place
    const T* fat = nullptr;    // its next vector
    int fleft = 0, foff = 0;   // places left of the share, empty ones before the next vector
    uint32_t put;              // this thread's place in the slot that is filled next, and in the tile last taken
    uint32_t got;
    const uint32_t begin, end;

    __device__ __forceinline__ Feed(const StatsArgs& args, uint4* smem, int group, int groups, int r, int c, int t)
        : a(args), ngroups(groups), rank(r), clog(c), tid(t), alike((args.ld * int(sizeof(T))) % 128 == 0),
          first(static_cast<const T*>(args.x), args.vocab, r, c), fr(group - groups),
          fynext(args.target && group < args.rows ? args.target[group] : 0), ring(smem + t),
          begin(static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + 16u * uint32_t(t)), end(begin + 16u * ST * tile) {
        put = begin;
        got = end - 16u * tile;
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) fetch();
    }
    __device__ __forceinline__ const T* row_at(int64_t r) const { return static_cast<const T*>(a.x) + r * a.ld; }
    __device__ __forceinline__ Place<T> place_of(const T* x) const { return alike ? first : Place<T>(x, a.vocab, rank, clog); }
    __device__ __forceinline__ void edge_tile() {   // a row's first or last tile
        while (fleft <= 0) {   // the next row that is not ignored and of which this CTA has a share
            fr += ngroups;
            if (fr >= a.rows) return;   // behind the last row a copy group is empty
            const int64_t y = fynext;
            if (a.target && fr + ngroups < a.rows) fynext = a.target[fr + ngroups];
            if (y < 0) continue;
            const T* const x = row_at(fr);
            const Place<T> pl = place_of(x);
            foff = pl.off;
            fleft = pl.hi > pl.lo ? pl.hi - pl.lo + pl.off : 0;
            fat = x + pl.head + int64_t(pl.lo + tid - pl.off) * N;
        }
#pragma unroll
        for (int i = 0; i < TV; ++i)
            if (tid + B * i < fleft && (i > 0 || tid >= foff)) copy_async(put + 16u * B * i, fat + B * N * i);
        if (tid < foff) ring[(put - begin) / 16] = make_uint4(Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty);
        foff = 0;
    }
    __device__ __forceinline__ void fetch() {
        if (fleft >= tile) {
#pragma unroll
            for (int i = 0; i < TV; ++i) copy_async(put + 16u * B * i, fat + B * N * i);
        } else {
            edge_tile();
        }
        copy_commit();
        fat += tile * N;
        fleft -= tile;
        put += 16u * tile;
        if (put == end) put = begin;
    }
    // The next tile; the one before is done with, its slot is the next to fill.
    __device__ __forceinline__ const uint4* take() {
        fetch();
        copy_wait<ST - 1>();
        got += 16u * tile;
        if (got == end) got = begin;
        return ring + (got - begin) / 16;
    }
};
// Four of a tile's vectors, from the g-th on, for a thread that has `mine` places left in it.
template <typename T, int B> __device__ __forceinline__ void load_four(const uint4* buf, int g, int mine, uint4 (&raw)[4]) {
    if (B * (g + 3) < mine) {
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = buf[B * (g + i)];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            raw[i] = make_uint4(Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty);
            if (B * (g + i) < mine) raw[i] = buf[B * (g + i)];
        }
    }
}

// The largest k entries without a second pass over the row.  The row's vectors fall into groups (a
// thread's consecutive ones) whose maxima the softmax's pass gives for nothing.  Let t be the k-th
// largest of these maxima: k groups have an entry >= t each, so every one of the k largest entries is
// >= t, and lies in a group whose maximum is.  Those groups (k, and a few that the search for t leaves)
// are read again, out of L2, their entries >= t are the candidates, which are put in
// order.  Where more candidates come together than fit (thousands of equal entries, or
// the largest ones side by side in a few groups), the exact k-th entry is searched for in the row itself.

// Vectors in a group: the least power of two with which `most` of them are at most `groups` groups.
__device__ __forceinline__ int group_shift(int most, int groups) {
    int gs = 0;
    while (groups << gs < most) ++gs;
    return gs;
}
// The maxima of a thread's groups, from four vectors at a time: those from vector `at` on.
template <typename T, int B, typename GT>
__device__ __forceinline__ float keep_maxima(GT (*gm)[B], int gs, int at, const uint4 (&raw)[4], float& run, int tid) {
    if (gs >= 2) {
        const float t = top_of<T>(raw);
        run = (at & ((1 << gs) - 1)) == 0 ? t : fmaxf(run, t);
        gm[at >> gs][tid] = from_f<GT>(run);
        return t;
    }
    float tops[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) tops[i] = Vec<T>::top(raw[i]);
    const float t01 = fmaxf(tops[0], tops[1]), t23 = fmaxf(tops[2], tops[3]);
    if (gs == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) gm[at + i][tid] = from_f<GT>(tops[i]);
    } else {
        gm[at >> 1][tid] = from_f<GT>(t01);
        gm[(at >> 1) + 1][tid] = from_f<GT>(t23);
    }
    return fmaxf(t01, t23);
}
__device__ __forceinline__ float lg2(float v) {
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// Of `sets` numbers at least k are >= the value of rank lo, and M is the largest: lo raised until few more
// than k are.  count(value): how many are >= it.  The logarithm of that count falls about evenly towards
// the largest ones: two steps of three go where it would be just above k, the third halves the ranks.
template <typename T, typename F>
__device__ __forceinline__ uint32_t search_rank(uint32_t lo, int sets, float M, int k, F count) {
    constexpr int SH = Order<T>::kShift;
    const int enough = k + k / 4 + 4;
    const float aim = lg2(1.1f * float(k) + 1.0f);
    uint32_t hi = rank_of<T>(M) + 1;
    float from = logit_of(lo << SH), to = M, lfrom = lg2(float(sets)), lto = 0.0f;   // the ends, and log2 of their counts
    for (int step = 0; hi - lo > 1; step = step == 2 ? 0 : step + 1) {
        uint32_t mid = lo + (hi - lo) / 2;
        if (step < 2) {
            const uint32_t guess = rank_of<T>(__fmaf_rn(to - from, (lfrom - aim) / (lfrom - lto), from));
            mid = guess > lo && guess < hi ? guess : mid;
        }
        const float v = logit_of(mid << SH);
        const int n = count(v);
        if (n < k) {
            hi = mid;
            to = v;
            lto = lg2(fmaxf(float(n), 1.0f));
            continue;
        }
        lo = mid;
        from = v;
        lfrom = lg2(float(n));
        if (n <= enough) break;
    }
    return lo;
}
// The entries >= least of NV vectors (at(i): the first element's id, below 0 for none) to the list:
// add(count) gives the place of a thread's first one, store(place, candidate) puts it there.
template <typename T, int NV, typename At, typename A, typename S>
__device__ __forceinline__ void offer_vectors(const uint4 (&raw)[NV], float least, At at, A add, S store) {
    constexpr int N = Vec<T>::N;
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (at(i) < 0 || !(Vec<T>::top(raw[i]) >= least)) continue;
        float f[N];
        Vec<T>::wide(raw[i], f);
#pragma unroll
        for (int j = 0; j < N; ++j) n += f[j] >= least;
    }
    if (n == 0) return;
    int to = add(n);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (at(i) < 0 || !(Vec<T>::top(raw[i]) >= least)) continue;
        float f[N];
        Vec<T>::wide(raw[i], f);
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (f[j] >= least) store(to++, candidate(order_of(f[j]), at(i) + j));
    }
}

// Vectors with an entry to be offered, side by side in shared memory, so that the threads share their
// entries evenly.
struct Stage {
    uint4* raw;
    int *id, *count;   // of a vector's first element
};
// Places for a thread's n, behind those that *count has already.
__device__ __forceinline__ int places_for(int n, int* count) { return n > 0 ? atomicAdd(count, n) : 0; }
// A thread's vectors `pass` (a bit each), of the first element's id id(i).
template <int NV, typename Id>
__device__ __forceinline__ void stage_vectors(const uint4 (&raw)[NV], unsigned pass, Id id, const Stage& st) {
    int to = places_for(__popc(pass), st.count);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (pass >> i & 1) {
            st.raw[to] = raw[i];
            st.id[to] = id(i);
            ++to;
        }
}
// The staged vectors' entries >= least to the list, by SB threads.
template <typename T, int SB, int CAP>
__device__ __forceinline__ void offer_staged(const Stage& st, int m, float least, unsigned long long* found, int* nfound, int tid) {
    constexpr int N = Vec<T>::N;
    for (int base = tid & ~31; base < m; base += SB) {
        const int i = base + (tid & 31);
        unsigned some = 0;
        int id = 0;
        if (i < m) {
            float f[N];
            Vec<T>::wide(st.raw[i], f);
            id = st.id[i];
#pragma unroll
            for (int j = 0; j < N; ++j) some |= f[j] >= least ? 1u << j : 0u;
        }
        int to = places_for(__popc(some), nfound);
        for (; some != 0 && to < CAP; some &= some - 1) {
            const int j = __ffs(some) - 1;
            found[to++] = candidate(order_of(to_f(reinterpret_cast<const T*>(st.raw + i)[j])), id + j);
        }
    }
}

// ---------------------------------------------------------------------------
// A CTA per row: warps that read rows, and warps that choose entries
// ---------------------------------------------------------------------------

constexpr int kList = 1024;   // groups that are read again; more: the exact search

// Dynamic shared memory of a CTA.  The maxima of a thread's 16 groups of vectors, and the largest of all,
// are kept in the logits' own type.
// A buffer belongs to one team (their number is a multiple of the teams'): a team that runs ahead of another
// would else take the other's rows for its own.
template <typename T, int B, int NT, int TV, int ST> struct TopShared {
    static constexpr int G = 16, NB = 2 * NT;
    uint4 ring[ST][TV * B];
    unsigned long long found[NT][kCandidates];
    T gmax[NB][G + 1][B];   // per buffer
    int bins[NT][kBins];
    uint16_t list[NT][kList];
};

// B threads read rows and leave the maxima of groups; NT teams of SB threads take rows in turns and
// choose their entries while the former are in the next rows.  NB rows' maxima are kept (`buffer`).
// Named barriers 1 + buffer: a row's maxima and sums are there; 1 + NB + buffer: they have been used;
// then one per team.
//
// What bounds it: the reading warps' instructions (four such warps to a scheduler, 59 % of the issue slots busy) and
// the second look, a tenth of whose lines have left L2.  4,096 x 128,256 bf16, all rows valid: 170 us with 1
// alternative, 199 with 64, 348 with 256 (the rows alone 155 at the copy rate); 2,048 of fp32 182 with 64.  Shorter
// rows are bound by the two teams: 4,096 x 50,001 bf16 122 with 64 (66 without alternatives), 8,192 x 32,003 195 (86).  Measured
// against it with 64: one team of four warps 206, 512 reading threads and teams of four 222, all warps choosing
// between rows 266; full tiles without guards 219 (more code than the instruction caches hold).
template <typename T, int B, int SB, int NT, int TV, int ST, int PER_SM>
__global__ void __launch_bounds__(B + NT * SB, PER_SM) k_top(const StatsArgs a) {
    using Shared = TopShared<T, B, NT, TV, ST>;
    constexpr int N = Vec<T>::N, nw = B / 32, G = Shared::G, NB = Shared::NB, HELD = B / SB, KEYS = HELD * 2, LOADS = 8;
    static_assert(nw <= 16 && 2 * NB + NT < 16, "parts of a row for half a warp, 16 named barriers");
    static_assert(kMaxAlternatives <= B, "every thread's half of a row is a set of its own");
    __shared__ float4 wparts[NB][nw];
    __shared__ int counts[NT][2][8], nfound[NT], nlist[NT], nstage[NT];
    extern __shared__ __align__(128) uint4 ring[];
    Shared& sh = *reinterpret_cast<Shared*>(ring);
    const int lane = threadIdx.x & 31;
    const float c2 = a.c2;
    const int group = blockIdx.x, ngroups = gridDim.x;
    int buffer = 0;
    auto next = [&]() { buffer = buffer + 1 == NB ? 0 : buffer + 1; };
    int64_t ynext = a.target && group < a.rows ? a.target[group] : 0;
    auto label = [&](int64_t r) {
        const int64_t y = ynext;
        if (a.target && r + ngroups < a.rows) ynext = a.target[r + ngroups];
        return y;
    };
    if (threadIdx.x < B) {
        // ------------------------------------------------------------ the rows
        const int tid = threadIdx.x, warp = tid >> 5;
        Feed<T, B, TV, ST> feed(a, ring, group, ngroups, 0, 0, tid);
        const Scale scale(a);
        int done = 0;   // rows so far, up to NB
        for (int64_t r = group; r < a.rows; r += ngroups) {
            if (label(r) < 0) continue;
            const T* const x = feed.row_at(r);
            const Place<T> pl = feed.place_of(x);
            const bool edge = tid < pl.edges;
            const float xe = edge ? to_f(x[pl.edge_at(tid)]) : kNegInf;
            const int places = pl.hi > pl.lo ? pl.hi - pl.lo + pl.off : 0;
            const int gs = group_shift((places + TV * B - 1) / (TV * B) * TV, G);
            if (done == NB) bar_sync(1 + NB + buffer, B + SB); else ++done;
            T(*const gm)[B] = sh.gmax[buffer];
#pragma unroll
            for (int g = 0; g < G; ++g) gm[g][tid] = from_f<T>(kNegInf);
            Running<T> sum;
            float top = kNegInf, run = kNegInf;
            for (int base = 0; base * B < places; base += TV) {
                const uint4* const buf = feed.take();
                const int mine = places - base * B - tid;
#pragma unroll 1
                for (int g = 0; g < TV; g += 4) {
                    if (B * g >= mine) break;
                    uint4 raw[4];
                    load_four<T, B>(buf, g, mine, raw);
                    const float t = keep_maxima<T, B, T>(gm, gs, base + g, raw, run, tid);
                    top = fmaxf(top, t);
                    sum.raise(t, c2);
                    sum.template add<true>(raw, B * (g + 3) < mine, scale);
                }
            }
            gm[G][tid] = from_f<T>(top);
            const float4 part = warp_part(sum, top, xe, edge, scale);
            if (lane == 0) wparts[buffer][warp] = part;
            bar_arrive(1 + buffer, B + SB);
            next();
        }
        // the teams' last rows
        for (int i = 0; i < done; ++i) {
            buffer = buffer == 0 ? NB - 1 : buffer - 1;
            bar_sync(1 + NB + buffer, B + SB);
        }
        copy_wait<0>();
        return;
    }
    // ---------------------------------------------------------------- the entries
    const int team = (threadIdx.x - B) / SB, tid = (threadIdx.x - B) % SB, warp = tid >> 5, bar = 1 + 2 * NB + team;
    const bool alike = (a.ld * int(sizeof(T))) % 128 == 0;
    const Place<T> first(static_cast<const T*>(a.x), a.vocab, 0, 0);
    unsigned long long* const found = sh.found[team];
    uint16_t* const list = sh.list[team];
    int turn = 0, whose = NT - 1;
    for (int64_t r = group; r < a.rows; r += ngroups, next()) {
        int64_t y = label(r);
        for (; y < 0 && r < a.rows; r += ngroups, y = r < a.rows ? label(r) : 0)
            if (team == 0) ignored_row(a, r, tid, SB);
        if (r >= a.rows) break;
        whose = whose + 1 == NT ? 0 : whose + 1;
        if (whose != team) continue;
        const T* const x = static_cast<const T*>(a.x) + r * a.ld;
        const Place<T> pl = alike ? first : Place<T>(x, a.vocab, 0, 0);
        const bool edge = tid < pl.edges;
        const float xe = edge ? to_f(x[pl.edge_at(tid)]) : kNegInf;
        const float xy = warp == 0 && a.logp && y < a.vocab ? to_f(x[y]) : 0.0f;
        const int places = pl.hi > pl.lo ? pl.hi - pl.lo + pl.off : 0;
        const int gs = group_shift((places + TV * B - 1) / (TV * B) * TV, G);
        const T(*const gm)[B] = sh.gmax[buffer];
        if (tid == 0) nfound[team] = nlist[team] = 0;
        bar_sync(1 + buffer, B + SB);
        const RowSums sums = join_parts<nw>(lane < nw ? wparts[buffer][lane] : make_float4(kNegInf, 0.0f, 0.0f, INFINITY), c2);
        const RowSoftmax row(sums, a, sizeof(T) == 4);
        if (warp == 0) row.finish(a, r, y, xy);
        if (row.none) {
            for (int i = tid; i < a.k; i += SB) put_entry(a, r, i, -1, row.share(0.0f));
            bar_arrive(1 + NB + buffer, B + SB);
            continue;
        }
        // The sets among which t is searched: the threads' vectors as wholes while there are twice as many
        // as k (the k largest of 4 k sets have 1.15 k entries >= t, of 2 k 1.39 k), else halves of them.
        const bool halves = 2 * a.k > B;
        float key[KEYS];   // of HELD threads
#pragma unroll
        for (int i = 0; i < KEYS; ++i) key[i] = kNegInf;
        if (!halves) {
#pragma unroll
            for (int i = 0; i < HELD; ++i) key[i] = to_f(gm[G][tid + i * SB]);
        } else {
#pragma unroll
            for (int i = 0; i < HELD; ++i)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const int half = 2 * i + (g & 1);   // also where few groups are used
                    key[half] = fmaxf(key[half], to_f(gm[g][tid + i * SB]));
                }
        }
        auto count = [&](float v) {
            int c = 0;
            if (!halves) {
#pragma unroll
                for (int i = 0; i < HELD; ++i) c += key[i] >= v;
            } else {
#pragma unroll
                for (int i = 0; i < KEYS; ++i) c += key[i] >= v;
            }
            return sum_over<SB>(c, counts[team], turn, tid, bar);
        };
        uint32_t lo = kLeast<T>;
        const bool full = sums.least > kNegInf;   // each thread has a set from the least of their tops on
        if (full) lo = rank_of<T>(sums.least);
        const int from = full ? (halves ? 2 * B : B) : count(logit_of(lo << Order<T>::kShift));
        if (from > a.k) lo = search_rank<T>(lo, from, row.M, a.k, count);
        const float least = logit_of(lo << Order<T>::kShift);
        // the groups from there on
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            const int t = tid + h * SB;
            if (!(to_f(gm[G][t]) >= least)) continue;
            unsigned some = 0;
#pragma unroll
            for (int g = 0; g < G; ++g) some |= to_f(gm[g][t]) >= least ? 1u << g : 0u;
            int i = atomicAdd(&nlist[team], __popc(some));
            for (; some != 0 && i < kList; some &= some - 1) list[i++] = uint16_t((__ffs(some) - 1) * B + t);
        }
        if (edge && xe >= least) found[atomicAdd(&nfound[team], 1)] = candidate(order_of(xe), pl.edge_at(tid));
        sync<SB>(bar);
        const int groups = nlist[team], items = groups > kList ? 0 : groups << gs;
        // where the maxima have been: 4 SB vectors and their ids
        static_assert(80 * SB <= int(sizeof(sh.gmax[0])), "a round's vectors take the place of a row's maxima");
        uint4* const staged = reinterpret_cast<uint4*>(sh.gmax[buffer]);
        const Stage stage{staged, reinterpret_cast<int*>(staged + 4 * SB), &nstage[team]};
        for (int base = 0; base < items; base += LOADS * SB) {
            uint4 raw[LOADS];
            auto place_at = [&](int i) {   // the id of a vector's first element, below 0 for none
                const int item = base + tid + SB * i;
                if (item >= items) return -1;
                const int e = list[item >> gs], t = e & (B - 1);
                const int place = t + B * (((e / B) << gs) + (item & ((1 << gs) - 1)));
                return place >= pl.off && place < places ? pl.head + (pl.lo + place - pl.off) * N : -1;
            };
            unsigned there = 0;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int at = place_at(i);
                there |= at >= 0 ? 1u << i : 0u;
                if (at >= 0) raw[i] = ld16(x + at);
            }
#pragma unroll
            for (int h = 0; h < LOADS; h += 4) {
                if (base + SB * h >= items) break;
                if (tid == 0) nstage[team] = 0;
                const uint4 four[4] = {raw[h], raw[h + 1], raw[h + 2], raw[h + 3]};
                unsigned pass = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) pass |= (there >> (h + i) & 1) && Vec<T>::top(four[i]) >= least ? 1u << i : 0u;
                sync<SB>(bar);
                stage_vectors<4>(four, pass, [&](int i) { return place_at(h + i); }, stage);
                sync<SB>(bar);
                offer_staged<T, SB, kCandidates>(stage, nstage[team], least, found, &nfound[team], tid);
                sync<SB>(bar);
            }
        }
        bar_arrive(1 + NB + buffer, B + SB);   // the maxima have been used
        int n = nfound[team];
        if (n > kCandidates || groups > kList)
            n = exact_candidates<T, SB>(x, a.vocab, a.k, lo, row.M, found, &nfound[team], counts[team], turn, tid, bar);
        place_candidates<T, SB>(found, n, lo, row.M, a.k, sh.bins[team], list, tid, bar, [&](unsigned long long c, int place) {
            put_entry(a, r, place, int(~uint32_t(c)), row.share(logit_of(uint32_t(c >> 32))));
        });
        for (int i = n + tid; i < a.k; i += SB) put_entry(a, r, i, -1, kNegInf);
        sync<SB>(bar);   // before the next row's candidates
    }
}

template <typename T, int B, int SB, int NT, int TV, int ST, int PER_SM>
cudaError_t top_launch(const StatsArgs& a, int sms, GroupCache& cache, cudaStream_t s) {
    auto* kernel = k_top<T, B, SB, NT, TV, ST, PER_SM>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(B + NT * SB);
    cfg.dynamicSmemBytes = sizeof(TopShared<T, B, NT, TV, ST>);
    cfg.stream = s;
    int groups = 0;
    cudaError_t e = resident_groups(reinterpret_cast<const void*>(kernel), cfg, RowShape{B + NT * SB, 0}, sms, cache, groups);
    if (e != cudaSuccess) return e;
    cfg.gridDim.x = unsigned(groups < a.rows ? groups : a.rows);
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// ---------------------------------------------------------------------------
// Short rows, held in registers
// ---------------------------------------------------------------------------

// A team of W warps per row, four warps to a CTA or (W = 8) eight, NV vectors per thread.  The row is read
// once; the entries are chosen where it is.  What bounds it: a row's chain of latencies (load, sums, search, candidates,
// order) with few rows under way: with alternatives 20 per SM at 1,000 16-bit entries (one warp, 8 vectors), 6 at 8,192
// (two warps, 16 vectors), without them 24 and 8.  bf16, without / with 8 alternatives: 16,384 x 1,000 16 / 30 us (5 at the
// copy rate), 16,384 x 8,192 55 / 111 (40); fp16 16 / 34 and 53 / 128: with alternatives its forms spill 100 to 500 bytes
// per thread, of widened entries that the search among entries keeps.
template <typename T, int W, int NV, bool TOP>
__global__ void __launch_bounds__(W > 4 ? 32 * W : 128, W > 4 ? 2 : NV > 8 ? (TOP ? 3 : 4) : NV > 4 ? (TOP ? 5 : 6) : TOP ? 7 : 8) k_held(const StatsArgs a) {
    constexpr int N = Vec<T>::N, SB = 32 * W, TEAMS = W < 4 ? 4 / W : 1, CAP = W == 1 ? 512 : kCandidates;
    __shared__ float4 wparts_of[TEAMS][2][W];   // by row parity
    __shared__ float2 wtops_of[TEAMS][2][W];
    __shared__ int counts_of[TEAMS][2][8], nfound[TEAMS], nstage[TEAMS];
    __shared__ __align__(16) int bins[TOP ? TEAMS : 1][kBins];
    extern __shared__ __align__(128) uint4 ring[];
    const int lane = threadIdx.x & 31, team = threadIdx.x / SB, tid = threadIdx.x % SB, warp = tid >> 5, bar = 1 + team;
    float4(*const wparts)[W] = wparts_of[team];
    float2(*const wtops)[W] = wtops_of[team];
    int(*const counts)[8] = counts_of[team];
    // per team: the staged vectors and their ids, and the candidates
    const Stage stage{ring + team * (SB * NV), reinterpret_cast<int*>(ring + TEAMS * SB * NV) + team * (SB * NV), &nstage[team]};
    unsigned long long* const found = reinterpret_cast<unsigned long long*>(reinterpret_cast<int*>(ring + TEAMS * SB * NV) + TEAMS * SB * NV) + team * CAP;
    const float c2 = a.c2;
    const Scale scale(a);
    const int64_t step = int64_t(gridDim.x) * TEAMS, start = int64_t(blockIdx.x) * TEAMS + team;
    int64_t ynext = a.target && start < a.rows ? a.target[start] : 0;
    int turn = 0, par = 0;
    for (int64_t r = start; r < a.rows; r += step) {
        const int64_t y = ynext;
        if (a.target && r + step < a.rows) ynext = a.target[r + step];
        if (y < 0) {
            ignored_row(a, r, tid, SB);
            continue;
        }
        const T* const x = static_cast<const T*>(a.x) + r * a.ld;
        const Place<T> pl(x, a.vocab, 0, 0);
        const T* const body = x + pl.head;
        const bool edge = tid < pl.edges;
        uint4 raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * SB + tid - pl.off;
            raw[i] = make_uint4(Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty);
            if (v >= 0 && v < pl.body) raw[i] = ld16(body + v * N);
        }
        const float xe = edge ? to_f(x[pl.edge_at(tid)]) : kNegInf;
        const float xy = a.logp && y < a.vocab ? to_f(x[y]) : 0.0f;
        float tops[NV], top = kNegInf, low = INFINITY;   // low: the least of the vectors' largest entries
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            top = fmaxf(top, tops[i] = Vec<T>::top(raw[i]));
            const int v = i * SB + tid - pl.off;
            if (TOP && v >= 0 && v < pl.body) low = fminf(low, tops[i]);
        }
        float M = warp_max(fmaxf(top, xe));
        if (TOP) low = -warp_max(-low);
        if (W > 1) {
            if (lane == 0) wtops[par][warp] = make_float2(M, low);
            sync<SB>(bar);
            // behind this barrier every warp has read the last row's count; the one of wparts comes before its use
            if (TOP && tid == 0) nfound[team] = nstage[team] = 0;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                M = fmaxf(M, wtops[par][i].x);
                low = fminf(low, wtops[par][i].y);
            }
        } else if (TOP) {
            if (lane == 0) nfound[team] = nstage[team] = 0;
            __syncwarp();
        }
        Running<T> sum;
        sum.raise(M, c2);
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
            const uint4 four[4] = {raw[i], raw[i + 1], raw[i + 2], raw[i + 3]};
            sum.template add<false>(four, false, scale);
        }
        sum.retake(top, scale);
        if (edge) sum.add_one(xe, scale);
        RowSums sums{M, warp_sum(sum.s), warp_sum(sum.w), kNegInf};
        if (W > 1) {
            if (lane == 0) wparts[par][warp] = make_float4(0.0f, sums.S, sums.W, 0.0f);
            sync<SB>(bar);
            sums.S = sums.W = 0.0f;
#pragma unroll
            for (int i = 0; i < W; i += 2) {
                sums.S += wparts[par][i].y + wparts[par][i + 1].y;
                sums.W += wparts[par][i].z + wparts[par][i + 1].z;
            }
            par ^= 1;
        }
        const RowSoftmax row(sums, a, sizeof(T) == 4);
        const bool finishes = warp == 0;
        if (!TOP || row.none) {
            if (finishes) row.finish(a, r, y, xy);
            if (TOP)
                for (int i = tid; i < a.k; i += SB) put_entry(a, r, i, -1, row.share(0.0f));
            continue;
        }
        // t among the vectors' maxima while there are twice as many as k, else among the entries themselves
        uint32_t lo = kLeast<T>;
        if (2 * a.k <= pl.body) {
            auto count = [&](float v) {
                int c = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) c += tops[i] >= v;
                return sum_over<SB>(c, counts, turn, tid, bar);
            };
            const bool full = low > kNegInf;
            if (full) lo = rank_of<T>(low);
            const int from = full ? pl.body : count(logit_of(lo << Order<T>::kShift));
            if (from > a.k) lo = search_rank<T>(lo, from, M, a.k, count);
        } else {
            auto count = [&](float v) {
                int c = xe >= v;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float f[N];
                    Vec<T>::wide(raw[i], f);
#pragma unroll
                    for (int j = 0; j < N; ++j) c += f[j] >= v;
                }
                return sum_over<SB>(c, counts, turn, tid, bar);
            };
            const int from = count(logit_of(lo << Order<T>::kShift));
            if (from > a.k) lo = search_rank<T>(lo, from, M, a.k, count);
        }
        const float least = logit_of(lo << Order<T>::kShift);
        if (edge && xe >= least) found[atomicAdd(&nfound[team], 1)] = candidate(order_of(xe), pl.edge_at(tid));
        unsigned pass = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) pass |= tops[i] >= least ? 1u << i : 0u;
        stage_vectors<NV>(raw, pass, [&](int i) { return pl.head + (i * SB + tid - pl.off) * N; }, stage);
        sync<SB>(bar);
        offer_staged<T, SB, CAP>(stage, nstage[team], least, found, &nfound[team], tid);
        sync<SB>(bar);
        int n = nfound[team];
        if (n > CAP) n = exact_candidates<T, SB>(x, a.vocab, a.k, lo, M, found, &nfound[team], counts, turn, tid, bar);
        place_candidates<T, SB>(found, n, lo, M, a.k, bins[team], reinterpret_cast<uint16_t*>(stage.raw), tid, bar, [&](unsigned long long c, int place) {
            put_entry(a, r, place, int(~uint32_t(c)), row.share(logit_of(uint32_t(c >> 32))));
        });
        for (int i = n + tid; i < a.k; i += SB) put_entry(a, r, i, -1, kNegInf);
        if (finishes) row.finish(a, r, y, xy);
        if (W == 1) __syncwarp();   // before the next row's counts; with more warps its first barrier comes before them
    }
}

template <typename T, int W, int NV, bool TOP>
cudaError_t held_launch(const StatsArgs& a, int sms, GroupCache& cache, cudaStream_t s) {
    auto* kernel = k_held<T, W, NV, TOP>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    constexpr int threads = W > 4 ? 32 * W : 128, rows = W < 4 ? 4 / W : 1;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = TOP ? size_t(8) * rows * (W == 1 ? 512 : kCandidates) + size_t(20) * NV * threads : 0;
    cfg.stream = s;
    int groups = 0;
    cudaError_t e = resident_groups(reinterpret_cast<const void*>(kernel), cfg, RowShape{threads, 0}, sms, cache, groups);
    if (e != cudaSuccess) return e;
    const int64_t want = (a.rows + rows - 1) / rows;
    cfg.gridDim.x = unsigned(groups < want ? groups : want);
    return cudaLaunchKernelEx(&cfg, kernel, a);
}
// As few warps to a row as hold it with 16 vectors per thread where there are rows for all of them, else more with
// fewer vectors.  us, bf16, one warp with 16 vectors / four with 4: 16,384 x 2,001 with 8 alternatives 54 / 82, without 26 / 38,
// 1,000 x 3,001 with 8 6.4 / 7.4, 300 x 3,001 5.8 / 5.1 (two warps with 8: 70, 33 and 6.8 of the first three); two warps with 16 /
// four with 8: 16,384 x 8,192 with 8 109 / 118, with 64 143 / 151, 1,000 x 8,192 with 8 11.0 / 10.7.
template <typename T, bool TOP> cudaError_t held(const StatsArgs& a, int places, int sms, GroupCache& cache, cudaStream_t s) {
    if (places <= 128) return held_launch<T, 1, 4, TOP>(a, sms, cache, s);
    if (places <= 256) return held_launch<T, 1, 8, TOP>(a, sms, cache, s);
    if (places <= 512) return a.rows > 4 * sms ? held_launch<T, 1, 16, TOP>(a, sms, cache, s) : held_launch<T, 4, 4, TOP>(a, sms, cache, s);
    if (places <= 1024) return a.rows > 8 * sms ? held_launch<T, 2, 16, TOP>(a, sms, cache, s) : held_launch<T, 4, 8, TOP>(a, sms, cache, s);
    if (places <= 2048) return held_launch<T, 4, 16, TOP>(a, sms, cache, s);
    return held_launch<T, 8, 16, TOP>(a, sms, cache, s);
}

// ---------------------------------------------------------------------------
// A group of CTAs per row
// ---------------------------------------------------------------------------

// Without alternatives: a group of 2^clog CTAs takes one row at a time, each CTA a contiguous share of the
// row's vectors.  What bounds it: memory (4,096 x 128,256 bf16: 148 us, 7.1 TB/s of reads; one row 4.9 us).
template <typename T, int B>
__global__ void __launch_bounds__(B, 512 / B) k_stats(const StatsArgs a, const int clog) {
    constexpr int TV = 8, ST = 3, nw = B / 32;
    __shared__ float4 wparts[2][8], cparts[2][kMaxCluster];   // by row parity: of the warps, of the CTAs
    extern __shared__ __align__(128) uint4 ring[];   // [ST][TV * B]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = 1 << clog, rank = cluster > 1 ? int(cluster_rank()) : 0;
    const int group = int(blockIdx.x) >> clog, ngroups = int(gridDim.x) >> clog;
    const float c2 = a.c2;
    const Scale scale(a);
    const float4 none_part = make_float4(kNegInf, 0.0f, 0.0f, INFINITY);
    Feed<T, B, TV, ST> feed(a, ring, group, ngroups, rank, clog, tid);
    if (cluster > 1) {   // every CTA of the group runs before any writes into another
        cluster_arrive();
        cluster_wait();
    }
    int par = 0, finisher = 0;
    int64_t ynext = a.target && group < a.rows ? a.target[group] : 0;
    for (int64_t r = group; r < a.rows; r += ngroups) {
        const int64_t y = ynext;
        if (a.target && r + ngroups < a.rows) ynext = a.target[r + ngroups];
        if (y < 0) {
            if (rank == 0) ignored_row(a, r, tid, B);
            continue;
        }
        const T* const x = feed.row_at(r);
        const Place<T> pl = feed.place_of(x);
        const bool edge = rank == 0 && tid < pl.edges;
        const float xe = edge ? to_f(x[pl.edge_at(tid)]) : kNegInf;
        // the warps take the rows' ends in turns
        const bool finishes = rank == 0 && warp == finisher;
        const float xy = finishes && a.logp && y < a.vocab ? to_f(x[y]) : 0.0f;
        const int places = pl.hi > pl.lo ? pl.hi - pl.lo + pl.off : 0;
        Running<T> sum;
        float top = kNegInf;
        for (int base = 0; base * B < places; base += TV) {
            const uint4* const buf = feed.take();
            const int mine = places - base * B - tid;
#pragma unroll 1
            for (int g = 0; g < TV; g += 4) {
                if (B * g >= mine) break;
                uint4 raw[4];
                load_four<T, B>(buf, g, mine, raw);
                const float t = top_of<T>(raw);
                top = fmaxf(top, t);
                sum.raise(t, c2);
                sum.template add<true>(raw, B * (g + 3) < mine, scale);
            }
        }
        const float4 part = warp_part(sum, top, xe, edge, scale);
        if (lane == 0) wparts[par][warp] = part;
        __syncthreads();
        if (cluster > 1) {
            if (warp == 0) {
                const RowSums p = join_parts<8>(lane < nw ? wparts[par][lane] : none_part, c2);
                if (lane < cluster) store_remote(&cparts[par][rank], uint32_t(lane), make_float4(p.M, p.S, p.W, p.least));
            }
            cluster_arrive();
            cluster_wait();
        }
        if (finishes) {
            const RowSums sums = cluster > 1 ? join_parts<8>(lane < cluster ? cparts[par][lane] : none_part, c2)
                                             : join_parts<8>(lane < nw ? wparts[par][lane] : none_part, c2);
            RowSoftmax(sums, a, sizeof(T) == 4).finish(a, r, y, xy);
        }
        par ^= 1;
        finisher = finisher + 1 == nw ? 0 : finisher + 1;
    }
    copy_wait<0>();
}

// With alternatives, for few rows: each CTA of the group chooses the k largest entries of its share and hands
// them, with its sums, to the first one, which puts all of them in order.  What bounds it: latency (one row of 128,256
// bf16 9.2 us with 20 alternatives, 4.9 without any).
constexpr int kJoined = 4096;   // candidates of all CTAs
template <int B> struct SpreadShared {
    static constexpr int G = 8;      // groups of vectors per thread
    uint4 ring[3][8 * B];
    unsigned long long found[kJoined];
    union {                          // the groups' maxima; then the share's candidates
        float gmax[G][B];
        unsigned long long home[G * B / 2];
    };
    uint16_t list[kJoined];          // groups to look at again; then the order of the candidates
};
template <typename T, int B>
__global__ void __launch_bounds__(B, 1) k_spread(const StatsArgs a, const int clog) {
    constexpr int TV = 8, ST = 3, nw = B / 32, G = SpreadShared<B>::G, kHome = G * B / 2, kPlaces = B * TV;
    static_assert(G * B <= kJoined, "every group has a place in the list");
    __shared__ float4 wparts[8], cparts[kMaxCluster];   // of the warps, of the CTAs
    __shared__ int counts[2][8], nfound, nlist, nhome, first_place;
    __shared__ __align__(16) int bins[kBins];
    extern __shared__ __align__(128) uint4 ring[];
    SpreadShared<B>& sh = *reinterpret_cast<SpreadShared<B>*>(ring);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = 1 << clog, rank = int(cluster_rank());
    const int group = int(blockIdx.x) >> clog, ngroups = int(gridDim.x) >> clog;
    const float c2 = a.c2;
    const Scale scale(a);
    const float4 none_part = make_float4(kNegInf, 0.0f, 0.0f, INFINITY);
    Feed<T, B, TV, ST> feed(a, ring, group, ngroups, rank, clog, tid);
    if (tid == 0) nfound = 0;
    cluster_arrive();   // every CTA of the group runs before any writes into another
    cluster_wait();
    int turn = 0;
    int64_t ynext = a.target && group < a.rows ? a.target[group] : 0;
    for (int64_t r = group; r < a.rows; r += ngroups) {
        const int64_t y = ynext;
        if (a.target && r + ngroups < a.rows) ynext = a.target[r + ngroups];
        if (y < 0) {
            if (rank == 0) ignored_row(a, r, tid, B);
            continue;
        }
        const T* const x = feed.row_at(r);
        const Place<T> pl = feed.place_of(x);
        const bool edge = rank == 0 && tid < pl.edges;
        const float xe = edge ? to_f(x[pl.edge_at(tid)]) : kNegInf;
        const float xy = rank == 0 && warp == 0 && a.logp && y < a.vocab ? to_f(x[y]) : 0.0f;
        const int places = pl.hi > pl.lo ? pl.hi - pl.lo + pl.off : 0;
        const int gs = group_shift((places + kPlaces - 1) / kPlaces * TV, G);
#pragma unroll
        for (int g = 0; g < G; ++g) sh.gmax[g][tid] = kNegInf;
        Running<T> sum;
        float top = kNegInf, run = kNegInf;
        const uint4* buf = nullptr;
        for (int base = 0; base * B < places; base += TV) {
            buf = feed.take();
            const int mine = places - base * B - tid;
#pragma unroll 1
            for (int g = 0; g < TV; g += 4) {
                if (B * g >= mine) break;
                uint4 raw[4];
                load_four<T, B>(buf, g, mine, raw);
                const float t = keep_maxima<T, B, float>(sh.gmax, gs, base + g, raw, run, tid);
                top = fmaxf(top, t);
                sum.raise(t, c2);
                sum.template add<true>(raw, B * (g + 3) < mine, scale);
            }
        }
        const float4 part = warp_part(sum, top, xe, edge, scale);
        if (lane == 0) wparts[warp] = part;
        if (tid == 0) nlist = nhome = 0;
        __syncthreads();
        const RowSums share = join_parts<8>(lane < nw ? wparts[lane] : none_part, c2);
        float key[G];
#pragma unroll
        for (int g = 0; g < G; ++g) key[g] = sh.gmax[g][tid];
        auto count = [&](float v) {
            int c = 0;
#pragma unroll
            for (int g = 0; g < G; ++g) c += key[g] >= v;
            return sum_over<B>(c, counts, turn, tid, 0);
        };
        uint32_t lo = kLeast<T>;
        if (share.M > kNegInf && share.M < INFINITY) {
            const bool full = a.k <= B && share.least > kNegInf;   // each thread has a group from the least of their tops on
            if (full) lo = rank_of<T>(share.least);
            const int from = full ? B * G : count(logit_of(lo << Order<T>::kShift));
            if (from > a.k) lo = search_rank<T>(lo, from, share.M, a.k, count);
        }
        const float least = logit_of(lo << Order<T>::kShift);
        if (top >= least) {
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (key[g] >= least) sh.list[atomicAdd(&nlist, 1)] = uint16_t(g * B + tid);
        }
        __syncthreads();
        auto add = [&](int n) { return atomicAdd(&nhome, n); };
        auto store = [&](int i, unsigned long long c) { if (i < kHome) sh.home[i] = c; };
        if (edge && xe >= least) store(add(1), candidate(order_of(xe), pl.edge_at(tid)));
        const int items = nlist << gs;
        const uint4* const tile = places <= kPlaces ? buf - tid : nullptr;   // a share of one tile is still there
        for (int first = tid; first < items; first += 4 * B) {
            uint4 raw[4];
            int at[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int item = first + B * i;
                at[i] = -1;
                if (item < items) {
                    const int e = sh.list[item >> gs], t = e & (B - 1);
                    const int place = t + B * (((e / B) << gs) + (item & ((1 << gs) - 1)));
                    if (place >= pl.off && place < places) {
                        at[i] = pl.head + (pl.lo + place - pl.off) * Vec<T>::N;
                        raw[i] = tile ? tile[place] : ld16(x + at[i]);
                    }
                }
            }
            offer_vectors<T, 4>(raw, least, [&](int i) { return at[i]; }, add, store);
        }
        __syncthreads();
        const int here = nhome;
        if (tid == 0 && here > 0) first_place = add_remote(remote_address(&nfound, 0), here <= kHome ? here : kJoined + 1);
        if (warp == 1 && lane == 0)
            store_remote(&cparts[rank], 0u, make_float4(share.M, share.S, share.W, __uint_as_float(lo)));
        __syncthreads();
        const uint32_t to = remote_address(sh.found, 0) + 8u * uint32_t(first_place);
        if (here > 0 && here <= kHome)
            for (int i = tid; i < here && first_place + i < kJoined; i += B) store_remote(to + 8u * uint32_t(i), sh.home[i]);
        cluster_arrive();
        cluster_wait();
        if (rank == 0) {
            const float4 p = lane < cluster ? cparts[lane] : make_float4(kNegInf, 0.0f, 0.0f, __uint_as_float(~0u));
            lo = __reduce_min_sync(~0u, p.x > kNegInf ? __float_as_uint(p.w) : ~0u);
            const RowSoftmax row(join_parts<8>(make_float4(p.x, p.y, p.z, 0.0f), c2), a, sizeof(T) == 4);
            if (row.none) {
                for (int i = tid; i < a.k; i += B) put_entry(a, r, i, -1, row.share(0.0f));
                __syncthreads();
            } else {
                int n = nfound;
                __syncthreads();
                if (n > kJoined) n = exact_candidates<T, B>(x, a.vocab, a.k, lo, row.M, sh.found, &nfound, counts, turn, tid, 0);
                place_candidates<T, B>(sh.found, n, lo, row.M, a.k, bins, sh.list, tid, 0, [&](unsigned long long c, int place) {
                    put_entry(a, r, place, int(~uint32_t(c)), row.share(logit_of(uint32_t(c >> 32))));
                });
                for (int i = n + tid; i < a.k; i += B) put_entry(a, r, i, -1, kNegInf);
            }
            if (warp == 0) row.finish(a, r, y, xy);
            if (tid == 0) nfound = 0;
        }
        if (r + ngroups < a.rows) {   // the first CTA has done with the row
            cluster_arrive();
            cluster_wait();
        }
    }
    copy_wait<0>();
}

template <typename T, int B, bool TOP>
cudaError_t stats_launch(const StatsArgs& a, int clog, int sms, GroupCache& cache, cudaStream_t s) {
    auto* kernel = TOP ? k_spread<T, B> : k_stats<T, B>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1u << clog);
    cfg.blockDim = dim3(B);
    cfg.dynamicSmemBytes = TOP ? sizeof(SpreadShared<B>) : size_t(16) * 3 * 8 * B;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << clog;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = clog > 0 ? 1 : 0;
    int groups = 0;
    cudaError_t e = resident_groups(reinterpret_cast<const void*>(kernel), cfg, RowShape{B, clog}, sms, cache, groups);
    if (e != cudaSuccess) return e;
    if (groups > a.rows) groups = int(a.rows);
    cfg.gridDim.x = unsigned(groups) << clog;
    return cudaLaunchKernelEx(&cfg, kernel, a, clog);
}

template <typename T>
cudaError_t stats(const StatsArgs& a, int sms, GroupCache& cache, cudaStream_t s) {
    const int vecs = (a.vocab + Vec<T>::N - 1) / Vec<T>::N, threads = vecs <= 8192 ? 128 : 256;
    // places of a row: its vectors, and the empty places before them (where all rows lie alike, theirs)
    const uintptr_t body = (reinterpret_cast<uintptr_t>(a.x) + 15) / 16;
    const int places = vecs + ((a.ld * int64_t(sizeof(T))) % 128 == 0 ? int(body & 7) : 7);
    // In registers up to 2,048 vectors, and up to 4,096 for rows that get a CTA each at once: us in registers / as below,
    // bf16: 16,384 x 8,192 with 64 alternatives 143 / 283, 4,096 x 12,000 with 8 62 / 75, without 26 / 27, 4,096 x 17,000 with
    // 8 104 / 84, without 49 / 34; 304 x 24,000 with 20 9.7 / 11.1, 600 x 24,000 with 20 18.2 / 15.0, 1 x 30,000 with 20
    // 7.1 / 9.0.
    if (places <= (a.rows <= 2 * sms ? 4096 : 2048)) return a.k > 0 ? held<T, true>(a, places, sms, cache, s) : held<T, false>(a, places, sms, cache, s);
    // few rows: spread each over more CTAs while the GPU has idle SMs and the share is over a tile
    int clog = 0;
    while (clog < kMaxClusterLog && a.rows << (clog + 1) <= sms && (threads * 8) << clog < vecs) clog += 1;
    if (a.k == 0) {
        if (threads == 128) return stats_launch<T, 128, false>(a, clog, sms, cache, s);
        return stats_launch<T, 256, false>(a, clog, sms, cache, s);
    }
    if (clog > 0) {
        if (threads == 128) return stats_launch<T, 128, true>(a, clog, sms, cache, s);
        return stats_launch<T, 256, true>(a, clog, sms, cache, s);
    }
    if constexpr (sizeof(T) == 4) return top_launch<T, 256, 64, 1, 4, 4, 2>(a, sms, cache, s);
    else return top_launch<T, 256, 64, 2, 4, 3, 2>(a, sms, cache, s);
}

// ---------------------------------------------------------------------------
// The gradient
// ---------------------------------------------------------------------------

// With q_j = 2^(w_j - rest) of the saved statistics,
//   dx_j = -step q_j (ga + gb (log q_j + H)) + [j = y] step ga = 2^w_j (A + B w_j) + [j = y] step ga:
// one exponential and four multiplications or additions per element, every element on its own.  One
// segment of a row per CTA.  What bounds it: memory (4,096 x 128,256 bf16, one row in eight ignored: 281 us, 7.0 TB/s;
// 1,500 x 32,003 fp32 55 us, 6.6 TB/s).
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
    const float c2 = a.c2, kNaN = __int_as_float(0x7fffffff);
    const float M = a.saved[3 * r], H = a.saved[3 * r + 2];
    const bool far = big(M, c2);
    const float u = far ? 0.0f : anchor(M, c2), base = far ? M : 0.0f;   // exponents are (v - base) c2 - u
    // log2 q_j = w_j - rest
    const float rest = __fmaf_rn(a.saved[3 * r + 1], kLog2e, far ? 0.0f : __fmaf_rn(M, c2, -u));
    const float step = (a.seed ? *a.seed : 1.0f) * a.it;
    const float ga = a.grad_logp ? a.grad_logp[r] : 0.0f, gb = a.grad_entropy ? a.grad_entropy[r] : 0.0f;
    const float scale = -step * ex2(-rest) + (y >= a.vocab ? kNaN : 0.0f);
    const float A = scale * __fmaf_rn(gb, __fmaf_rn(-rest, kLn2, H), ga), B = scale * gb * kLn2, at_label = step * ga;
    auto value = [&](float v) {
        const float w = fmaxf(__fmaf_rn(half_apart(v, base), 2.0f * c2, -u), kLowest);
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
