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

// log q of an entry x of a row with a softmax.  Roundings of the sum are not let above 0, and an entry at
// a type's lowest value, whose exponent overflows, has its distance.
__device__ __forceinline__ float log_q(float x, float M, float u, float c2, bool far, float S, float it) {
    const float r = log_share(x, M, u, c2, far, S);
    return fminf(r == kNegInf ? (x - M) * it : r, 0.0f);
}

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
// The larger of both, NaN if v is.
__device__ __forceinline__ float max_nan(float v, float least) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(least));
    return r;
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

constexpr int kGroups = 8;          // of vectors, per thread, over all CTAs of a row
constexpr int kCandidates = 1024;

// Other CTAs' shared memory.
__device__ __forceinline__ uint32_t remote_address(const void* smem, uint32_t rank) {
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(smem)), to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
    return to;
}
__device__ __forceinline__ void store_remote(uint32_t to, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
}
__device__ __forceinline__ void store_remote(uint32_t to, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(v) : "memory");
}
__device__ __forceinline__ int add_remote(uint32_t to, int v) {
    int r;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(to), "r"(v) : "memory");
    return r;
}

// What a row's sums amount to; by every lane of a warp, whose lanes 0 .. n - 1 (n <= 8) hold the parts
// (largest entry, S, W, and the least of the threads' largest entries).
struct RowSums {
    float M, S, W, least;
};
__device__ __forceinline__ RowSums join_parts(float4 p, float c2) {
    RowSums r;
    r.M = warp_max(p.x);
    r.least = -warp_max(-p.w);
    move_sums(p.x, part_ref(r.M), c2, p.y, p.z);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        p.y += __shfl_xor_sync(~0u, p.y, o);
        p.z += __shfl_xor_sync(~0u, p.z, o);
    }
    r.S = __shfl_sync(~0u, p.y, 0);
    r.W = __shfl_sync(~0u, p.z, 0);
    return r;
}

// ---------------------------------------------------------------------------
// A group of CTAs per row
// ---------------------------------------------------------------------------

constexpr int kTileVecs = 8, kStages = 3;

// A group of 2^clog CTAs takes one row at a time, each CTA a contiguous share of the row's vectors,
// which come through shared memory in tiles, copied asynchronously ahead of their use, the next row's
// too.  A thread copies the vectors that it will itself use.
//
// The largest k entries without a second pass over the row.  The row's vectors fall into groups (a
// thread's consecutive ones, eight groups to the threads of one place in the row's CTAs) whose maxima
// the softmax's pass gives for nothing.  Let t be the k-th largest of these maxima: k groups have an
// entry >= t each, so every one of the k largest entries is >= t, and lies in a group whose maximum is.
// Those groups (k, and a few that the search for t leaves) are read again, out of L2, their entries
// >= t are the candidates, and a candidate's place is the number of candidates before it.
//
// Where more candidates come together than fit (thousands of equal entries, or the largest ones side by
// side in a few groups), the exact k-th entry is searched for in the row itself: every count is a pass
// out of L2.
template <typename T, int B, bool TOP>
__global__ void __launch_bounds__(B, 512 / B) k_stats(const StatsArgs a, const int clog) {
    constexpr int N = Vec<T>::N, U = 4, tile = B * kTileVecs, ST = kStages, nw = B / 32, G = kGroups;
    __shared__ float4 wparts[2][8], cparts[2][kMaxCluster];   // by row parity: of the warps, of the CTAs
    __shared__ int counts[2][3][8], nfound[2], nlist[2];
    extern __shared__ __align__(128) uint4 ring[];   // [ST][tile]
    unsigned long long* const found = reinterpret_cast<unsigned long long*>(ring + ST * tile);   // [kCandidates]
    float(*const gmax)[B] = reinterpret_cast<float(*)[B]>(found + kCandidates);                   // [G][B]
    uint16_t* const list = reinterpret_cast<uint16_t*>(gmax);   // [G * B], where the maxima have been
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = 1 << clog, rank = cluster > 1 ? int(cluster_rank()) : 0;
    const int group = int(blockIdx.x) >> clog, ngroups = int(gridDim.x) >> clog;
    const int own = G >> clog;   // groups of this CTA's threads
    const float c2 = a.it * kLog2e, kNaN = __int_as_float(0x7fffffff);
    const pair_t c2c2 = pair_of(c2, c2);
    const uint4 empty = make_uint4(Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty, Vec<T>::kEmpty);
    const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + 16u * uint32_t(tid);
    auto row_at = [&](int64_t r) { return static_cast<const T*>(a.x) + r * a.ld; };
    // all rows lie alike where their stride is a multiple of 128 bytes
    const bool alike = (a.ld * int(sizeof(T))) % 128 == 0;
    const Place<T> first_place(static_cast<const T*>(a.x), a.vocab, rank, clog);
    auto place_of = [&](const T* x) { return alike ? first_place : Place<T>(x, a.vocab, rank, clog); };

    // The copies run ahead in the order of their use: the next vector of this thread, places left of the
    // share, empty places before the next vector.
    int64_t fr = group - ngroups, fynext = a.target && group < a.rows ? a.target[group] : 0;
    const T* fat = nullptr;
    int fleft = 0, foff = 0;
    auto fetch = [&](int slot) {
        while (fleft <= 0) {   // the next row that is not ignored and of which this CTA has a share
            fr += ngroups;
            if (fr >= a.rows) break;
            const int64_t y = fynext;
            if (a.target && fr + ngroups < a.rows) fynext = a.target[fr + ngroups];
            if (y < 0) continue;
            const T* const x = row_at(fr);
            const Place<T> pl = place_of(x);
            foff = pl.off;
            fleft = pl.hi > pl.lo ? pl.hi - pl.lo + pl.off : 0;
            fat = x + pl.head + int64_t(pl.lo + tid - pl.off) * N;
        }
        const uint32_t to = ring_at + 16u * uint32_t(slot * tile);
        if (fleft >= tile && foff == 0) {
#pragma unroll
            for (int i = 0; i < kTileVecs; ++i) copy_async(to + 16u * B * i, fat + B * N * i);
        } else {   // behind the last row a group is empty
#pragma unroll
            for (int i = 0; i < kTileVecs; ++i)
                if (tid + B * i < fleft && (i > 0 || tid >= foff)) copy_async(to + 16u * B * i, fat + B * N * i);
            if (tid < foff) ring[slot * tile + tid] = empty;
            foff = 0;
        }
        fat += tile * N;
        fleft -= tile;
        copy_commit();
    };
    int slot = -1;   // of the tile last taken
    auto take_tile = [&]() {   // the tile before is done with; its slot is the next to fill
        const int before = slot;
        slot = slot + 1 == ST ? 0 : slot + 1;
        fetch(before < 0 ? ST - 1 : before);
        copy_wait<ST - 1>();
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch(i);
    if (cluster > 1) {   // every CTA of the group runs before any writes into another
        cluster_arrive();
        cluster_wait();
    }

    int par = 0, turn = 0, finisher = 0;
    int64_t ynext = a.target && group < a.rows ? a.target[group] : 0;
    for (int64_t r = group; r < a.rows; r += ngroups) {
        const int64_t y = ynext;
        if (a.target && r + ngroups < a.rows) ynext = a.target[r + ngroups];
        auto put = [&](int i, int id, float lp) {
            const int64_t at = r * a.ld_top + i;
            if (a.id_bytes == 8) static_cast<int64_t*>(a.top_id)[at] = id; else static_cast<int32_t*>(a.top_id)[at] = id;
            a.top_logp[at] = lp;
        };
        if (y < 0) {
            if (rank == 0) {
                if (TOP)
                    for (int i = tid; i < a.k; i += B) put(i, -1, 0.0f);
                if (tid == 0) {
                    if (a.logp) a.logp[r] = 0.0f;
                    if (a.entropy) a.entropy[r] = 0.0f;
                }
                if (tid < 3 && a.saved) a.saved[3 * r + tid] = 0.0f;
            }
            continue;
        }
        const T* const x = row_at(r);
        const Place<T> pl = place_of(x);
        const bool edge = rank == 0 && tid < pl.edges;
        const float xe = edge ? to_f(x[pl.edge_at(tid)]) : kNegInf;
        // the warps take the rows' ends in turns
        const bool finishes = rank == 0 && warp == finisher;
        float xy = 0.0f;
        if (finishes && a.logp && y < a.vocab) xy = to_f(x[y]);
        // vectors of a group: the least power of two with which a thread's vectors are at most `own` groups
        const int places = pl.hi > pl.lo ? pl.hi - pl.lo + pl.off : 0;
        int gs = 0;
        if (TOP) {
            const int most = (places + tile - 1) / tile * kTileVecs;
            while (own << gs < most) ++gs;
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (g < own) gmax[rank * own + g][tid] = kNegInf;
        }
        // one pass: the largest entry, and the sums against a reference near it, U vectors at a time
        float top = kNegInf, m = kNegInf, s = 0.0f, w = 0.0f, run = kNegInf;
        for (int base = 0; base * B < places; base += kTileVecs) {
            take_tile();
            const uint4* const buf = ring + slot * tile + tid;
            const int mine = places - base * B - tid;
#pragma unroll 1
            for (int g = 0; g < kTileVecs; g += U) {
                if (B * g >= mine) break;
                uint4 raw[U];
                float tops[U];
                if (B * (g + U - 1) < mine) {
#pragma unroll
                    for (int i = 0; i < U; ++i) raw[i] = buf[B * (g + i)];
                } else {
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        raw[i] = empty;
                        if (B * (g + i) < mine) raw[i] = buf[B * (g + i)];
                    }
                }
#pragma unroll
                for (int i = 0; i < U; ++i) tops[i] = Vec<T>::top(raw[i]);
                const float t01 = fmaxf(tops[0], tops[1]), t23 = fmaxf(tops[2], tops[3]), t = fmaxf(t01, t23);
                if (TOP) {
                    float(*const gm)[B] = gmax + rank * own;
                    const int at = base + g;
                    if (gs == 0) {
#pragma unroll
                        for (int i = 0; i < U; ++i) gm[at + i][tid] = tops[i];
                    } else if (gs == 1) {
                        gm[at >> 1][tid] = t01;
                        gm[(at >> 1) + 1][tid] = t23;
                    } else {
                        run = (at & ((1 << gs) - 1)) == 0 ? t : fmaxf(run, t);
                        gm[at >> gs][tid] = run;
                    }
                }
                top = fmaxf(top, t);
                // smaller steps are left: m is a reference, and exponentials up to 2^32 of it do no harm
                if ((t - m) * c2 > 32.0f) {
                    move_sums(m, t, c2, s, w);
                    m = t;
                }
                const float ref = part_ref(m);
                if (big(ref, c2)) {
#pragma unroll 1
                    for (int i = 0; i < U * N && B * (g + i / N) < mine; ++i) {
                        const float v = to_f(reinterpret_cast<const T*>(buf + B * (g + i / N))[i % N]);
                        const float z = max_nan((v - ref) * c2, kLowest), e = ex2(z);
                        s += e;
                        w = __fmaf_rn(e, z, w);
                    }
                } else {
                    const float u = anchor(ref, c2);
                    const pair_t uu = pair_of(-u, -u);
                    pair_t s2 = 0, w2 = 0;   // of these vectors first: see tree_sum
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        float f[N];
                        Vec<T>::wide(raw[i], f);
#pragma unroll
                        for (int j = 0; j < N; j += 2) {
                            float z0, z1;
                            apart(fma_pair(pair_of(f[j], f[j + 1]), c2c2, uu), z0, z1);
                            z0 = max_nan(z0, kLowest);
                            z1 = max_nan(z1, kLowest);
                            const pair_t e = pair_of(ex2(z0), ex2(z1));
                            s2 = add_pair(s2, e);
                            w2 = fma_pair(e, pair_of(z0, z1), w2);
                        }
                    }
                    float p0, p1;
                    apart(s2, p0, p1);
                    s += p0 + p1;
                    apart(w2, p0, p1);
                    w += p0 + p1;
                }
            }
        }
        {
            // the warp's part, edges included
            const float wt = warp_max(fmaxf(top, xe)), ref = part_ref(wt), least = -warp_max(-top);
            move_sums(m, ref, c2, s, w);
            if (edge) {
                const float z = max_nan(big(ref, c2) ? (xe - ref) * c2 : __fmaf_rn(xe, c2, -anchor(ref, c2)), kLowest), e = ex2(z);
                s += e;
                w = __fmaf_rn(e, z, w);
            }
            s = warp_sum(s);
            w = warp_sum(w);
            if (lane == 0) wparts[par][warp] = make_float4(wt, s, w, least);
            if (tid == 0) nfound[par] = nlist[par] = 0;
        }
        const float4 none_part = make_float4(kNegInf, 0.0f, 0.0f, INFINITY);
        RowSums row;
        __syncthreads();
        if (cluster > 1) {
            if (warp == 0) {
                row = join_parts(lane < nw ? wparts[par][lane] : none_part, c2);
                if (lane < cluster) store_remote(&cparts[par][rank], uint32_t(lane), make_float4(row.M, row.S, row.W, row.least));
            }
            if (TOP)
                for (int c = 0; c < cluster; ++c) {
                    if (c == rank) continue;
                    for (int g = rank * own; g < (rank + 1) * own; ++g)
                        store_remote(remote_address(&gmax[g][tid], uint32_t(c)), gmax[g][tid]);
                }
            cluster_arrive();
            cluster_wait();
        }
        const int was = par;
        par ^= 1;
        if (TOP || finishes) {
            row = cluster > 1 ? join_parts(lane < cluster ? cparts[was][lane] : none_part, c2)
                              : join_parts(lane < nw ? wparts[was][lane] : none_part, c2);
        }
        finisher = finisher + 1 == nw ? 0 : finisher + 1;
        if (!TOP && !finishes) continue;
        const float M = row.M, S = row.S;
        const bool none = !(fabsf(M) < INFINITY) || S != S;   // no softmax
        const bool far = big(M, c2);
        const float u = anchor(M, c2);
        auto share = [&](float x) { return none ? kNaN : log_q(x, M, u, c2, far, S, a.it); };
        if (finishes) {
            const float log_sum = -share(M), lp = share(xy);
            const float H = fmaxf(log_sum + ((far ? 0.0f : __fmaf_rn(M, c2, -u)) - row.W / S) * kLn2, 0.0f);
            if (lane == 0) {
                if (a.logp) a.logp[r] = y < a.vocab ? lp : kNaN;
                if (a.entropy) a.entropy[r] = none ? kNaN : H;
                if (a.saved) {
                    a.saved[3 * r] = none ? kNaN : M;
                    a.saved[3 * r + 1] = log_sum;
                    a.saved[3 * r + 2] = none ? kNaN : H;
                }
            }
        }
        if (!TOP) continue;
        if (none) {
            if (rank == 0)
                for (int i = tid; i < a.k; i += B) put(i, -1, kNaN);
            continue;
        }
        // t: at least k groups are >= lo (or lo is the least), fewer than k are >= hi
        uint32_t key[G];
#pragma unroll
        for (int g = 0; g < G; ++g) key[g] = rank_of<T>(gmax[g][tid]);
        // how many groups are >= each of three ranks
        auto groups_from = [&](uint32_t t0, uint32_t t1, uint32_t t2, int (&n)[3]) {
            int c = 0;   // at most 8 per thread, 256 per warp: ten bits each
#pragma unroll
            for (int g = 0; g < G; ++g) c += (key[g] >= t0 ? 1 : 0) + (key[g] >= t1 ? 1 << 10 : 0) + (key[g] >= t2 ? 1 << 20 : 0);
            c = __reduce_add_sync(~0u, c);
            if (lane < 3) counts[turn][lane][warp] = (c >> (10 * lane)) & 0x3ff;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                n[i] = 0;
#pragma unroll
                for (int v = 0; v < nw; ++v) n[i] += counts[turn][i][v];
            }
            turn ^= 1;
        };
        // every thread that has a vector has a group from the least of their largest entries on
        const int enough = a.k + a.k / 2 + 16;
        uint32_t lo = kLeast<T>, hi = rank_of<T>(M) + 1;
        int over = G * B, n3[3];
        if (a.k <= B && row.least > kNegInf) {
            lo = rank_of<T>(row.least);
        } else {
            groups_from(lo, lo, lo, n3);
            over = n3[0];
        }
        while (over > enough && hi - lo > 1) {
            const uint32_t d = hi - lo, q = d >> 2, m0 = lo + q, m1 = lo + (d >> 1), m2 = hi - (q > 0 ? q : 1);
            groups_from(m0, m1, m2, n3);
            if (n3[2] >= a.k) { lo = m2; over = n3[2]; }
            else if (n3[1] >= a.k) { lo = m1; hi = m2; over = n3[1]; }
            else if (n3[0] >= a.k) { lo = m0; hi = m1; over = n3[0]; }
            else hi = m0;
        }
        // the groups from lo on, each CTA its own, and their entries from lo on, to the first CTA
        __syncthreads();
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int i = g - rank * own;
            if (i >= 0 && i < own && key[g] >= lo) list[atomicAdd(&nlist[was], 1)] = uint16_t(i * B + tid);
        }
        __syncthreads();
        const uint32_t far_found = cluster > 1 ? remote_address(found, 0) : 0, far_count = cluster > 1 ? remote_address(&nfound[was], 0) : 0;
        auto offer = [&](float v, int id) {
            const uint32_t o = order_of(v);
            if (o >> Order<T>::kShift < lo) return;
            if (cluster > 1) {
                const int i = add_remote(far_count, 1);
                if (i < kCandidates) store_remote(far_found + 8u * uint32_t(i), candidate(o, id));
            } else {
                const int i = atomicAdd(&nfound[was], 1);
                if (i < kCandidates) found[i] = candidate(o, id);
            }
        };
        if (edge) offer(xe, pl.edge_at(tid));
        const int items = nlist[was] << gs;
        for (int first = tid; first < items; first += B * U) {
            uint4 raw[U];
            int at[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int item = first + B * i;
                at[i] = -1;
                if (item < items) {
                    const int e = list[item >> gs], t = e & (B - 1);
                    const int place = t + B * (((e / B) << gs) + (item & ((1 << gs) - 1)));
                    if (place >= pl.off && place < places) at[i] = pl.lo + place - pl.off;
                }
                if (at[i] >= 0) raw[i] = ld16(x + pl.head + int64_t(at[i]) * N);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (at[i] < 0 || rank_of<T>(Vec<T>::top(raw[i])) < lo) continue;
                float f[N];
                Vec<T>::wide(raw[i], f);
#pragma unroll
                for (int j = 0; j < N; ++j) offer(f[j], pl.head + at[i] * N + j);
            }
        }
        if (cluster > 1) {
            cluster_arrive();
            cluster_wait();
            if (rank != 0) continue;
        } else {
            __syncthreads();
        }
        int n = nfound[was];
        if (n > kCandidates) {
            // the k-th largest entry itself: at least k entries are >= lo, fewer than k are >= hi
            auto entries_from = [&](uint32_t t) {
                int c = 0;
                for (int j = tid; j < a.vocab; j += B) c += rank_of<T>(to_f(x[j])) >= t;
                c = __reduce_add_sync(~0u, c);
                if (lane == 0) counts[turn][0][warp] = c;
                __syncthreads();
                c = 0;
#pragma unroll
                for (int v = 0; v < nw; ++v) c += counts[turn][0][v];
                turn ^= 1;
                return c;
            };
            hi = rank_of<T>(M) + 1;
            bool first = true;   // thousands of equal entries: the next rank already has fewer than k
            while (hi - lo > 1) {
                const uint32_t mid = first ? lo + 1 : lo + (hi - lo) / 2;
                first = false;
                if (entries_from(mid) >= a.k) lo = mid; else hi = mid;
            }
            __syncthreads();
            if (tid == 0) nfound[was] = 0;
            __syncthreads();
            for (int j = tid; j < a.vocab; j += B) {   // fewer than k
                const uint32_t o = order_of(to_f(x[j]));
                if (o >> Order<T>::kShift > lo) found[atomicAdd(&nfound[was], 1)] = candidate(o, j);
            }
            __syncthreads();
            n = nfound[was];
            // of those equal to the k-th the first ones
            for (int base = 0; n < a.k && base < a.vocab; base += B) {
                const int j = base + tid;
                const uint32_t o = j < a.vocab ? order_of(to_f(x[j])) : 0u;
                const bool equal = j < a.vocab && o >> Order<T>::kShift == lo;
                const unsigned ones = __ballot_sync(~0u, equal);
                if (lane == 0) counts[turn][0][warp] = __popc(ones);
                __syncthreads();
                int before = __popc(ones & ((1u << lane) - 1)), all = 0;
#pragma unroll
                for (int v = 0; v < nw; ++v) {
                    before += v < warp ? counts[turn][0][v] : 0;
                    all += counts[turn][0][v];
                }
                turn ^= 1;
                if (equal && n + before < a.k) found[n + before] = candidate(o, j);
                n += all;
            }
            n = min(n, a.k);
            __syncthreads();
        }
        // places: L lanes to a candidate where that keeps all of them busy at once
        const int ls = 4 * n <= B ? 2 : 2 * n <= B ? 1 : 0, part = tid & ((1 << ls) - 1);
        for (int i = tid >> ls; i < (n + 31 & ~31); i += B >> ls) {
            const unsigned long long c = i < n ? found[i] : 0;
            int place = 0;
#pragma unroll 4
            for (int j = part; j < n; j += 1 << ls) place += found[j] > c;
            if (ls > 0) place += __shfl_xor_sync(~0u, place, 1);
            if (ls > 1) place += __shfl_xor_sync(~0u, place, 2);
            if (part == 0 && i < n && place < a.k) put(place, int(~uint32_t(c)), share(logit_of(uint32_t(c >> 32))));
        }
        for (int i = n + tid; i < a.k; i += B) put(i, -1, kNegInf);
    }
    copy_wait<0>();
}

template <typename T, int B, bool TOP>
cudaError_t stats_launch(const StatsArgs& a, int clog, int sms, GroupCache& cache, cudaStream_t s) {
    auto* kernel = k_stats<T, B, TOP>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1u << clog);
    cfg.blockDim = dim3(B);
    cfg.dynamicSmemBytes = size_t(16) * kStages * kTileVecs * B + (TOP ? size_t(8) * kCandidates + size_t(4) * kGroups * B : 0);
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

template <typename T, bool TOP>
cudaError_t stats(const StatsArgs& a, int sms, GroupCache& cache, cudaStream_t s) {
    const int vecs = (a.vocab + Vec<T>::N - 1) / Vec<T>::N, threads = vecs < 512 ? 64 : vecs <= 8192 ? 128 : 256;
    // few rows: spread each over more CTAs while the GPU has idle SMs and the share is over a tile
    int clog = 0;
    while (clog < kMaxClusterLog && a.rows << (clog + 1) <= sms && (threads * kTileVecs) << clog < vecs) clog += 1;
    if (threads == 64) return stats_launch<T, 64, TOP>(a, clog, sms, cache, s);
    if (threads == 128) return stats_launch<T, 128, TOP>(a, clog, sms, cache, s);
    return stats_launch<T, 256, TOP>(a, clog, sms, cache, s);
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
    if (dt == kF32) return a.k > 0 ? stats<float, true>(a, sm_count, cache, s) : stats<float, false>(a, sm_count, cache, s);
    if (dt == kBF16) return a.k > 0 ? stats<__nv_bfloat16, true>(a, sm_count, cache, s) : stats<__nv_bfloat16, false>(a, sm_count, cache, s);
    return a.k > 0 ? stats<__half, true>(a, sm_count, cache, s) : stats<__half, false>(a, sm_count, cache, s);
}

cudaError_t launch_token_grad(int dt, const TokenGradArgs& a, cudaStream_t s) {
    if (dt == kF32) return token_grad<float>(a, s);
    if (dt == kBF16) return token_grad<__nv_bfloat16>(a, s);
    return token_grad<__half>(a, s);
}

}  // namespace tl
