// tl_dropout.cu - dropout whose mask is never stored (include/tl_dropout.h): the kernels, the checks
// of arguments and the launch.
//
// Mathematics.  Eight consecutive elements share one block of Philox4x32-10, 128 bits made of the
// block's number, the key that the device reads, and the site: 16 bits per element, compared with
// P = round(65536 p).  The number in the high half of a word w is >= P where w >= P << 16, that in
// the low half where w << 16 is: no number is taken out of its word.
#include "tl_loss_device.cuh"
#include "tl_spans.h"

#include <cmath>
#include <type_traits>

#include "../../include/tl_dropout.h"

namespace tl {
namespace {

struct DropoutArgs {
    const void* x;
    const void* residual;
    void* y;
    int64_t rows, cols, ldx, ldr, ldy;
    const int64_t* key;
    uint32_t site;
    uint32_t limit;      // P << 16; kept where a number is not below it
    bool random;         // else nothing is drawn: all numbers are 0
    float scale;         // 1 / (1 - P / 65536)
};

struct Philox {
    uint32_t k0, k1, ticket, above, site;
    __device__ __forceinline__ explicit Philox(const DropoutArgs& a) {
        const uint64_t seed = uint64_t(a.key[0]), t = uint64_t(a.key[1]);
        k0 = uint32_t(seed);
        k1 = uint32_t(seed >> 32);
        ticket = uint32_t(t);
        above = uint32_t(t >> 32) << 8;
        site = a.site;
    }
    // The four words of block b: ten rounds.
    __device__ __forceinline__ uint4 operator()(uint64_t b) const {
        uint32_t c0 = uint32_t(b), c1 = uint32_t(b >> 32) | above, c2 = ticket, c3 = site, q0 = k0, q1 = k1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p0 = uint64_t(c0) * 0xD2511F53u, p1 = uint64_t(c2) * 0xCD9E8D57u;
            c0 = uint32_t(p1 >> 32) ^ c1 ^ q0;
            c1 = uint32_t(p1);
            c2 = uint32_t(p0 >> 32) ^ c3 ^ q1;
            c3 = uint32_t(p0);
            q0 += 0x9E3779B9u;
            q1 += 0xBB67AE85u;
        }
        return make_uint4(c0, c1, c2, c3);
    }
};

__device__ __forceinline__ uint32_t word_of(const uint4& w, int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }

// Element `place` of a block.
__device__ __forceinline__ bool kept(uint32_t word, int place, uint32_t limit) {
    return (place & 1 ? word : word << 16) >= limit;
}
__device__ __forceinline__ float dropped(float x, bool keep, float scale, float residual) {
    return keep ? __fmaf_rn(x, scale, residual) : residual;
}

// Threads per CTA, and blocks of eight elements under way per thread.  us for 268M bf16 elements without a residual
// with 2 / 4 / 8 blocks and 128 threads: 160 / 152 / 186, with 4 and 256 threads 153; with a residual 224 with 1, 2 or 4;
// 8.4M elements with a residual 7.6 / 6.5 / 6.4 with 1 / 2 / 4, without one 6.4 / 6.1 / 7.1 with 2 / 4 / 8.  What bounds it: memory
// (152 us are 104 % of the copy rate, and 119 instructions for a thread's eight elements fill 70 % of the issue slots).
constexpr int kDropThreads = 128;
template <bool RES> constexpr int kBlocks = RES ? 2 : 4;

// Eight consecutive elements: one access of 16 bytes, or of 32 (fp32).
template <typename T> struct Eight {
    uint4 v;
    __device__ __forceinline__ void load(const T* p) { v = ld16(p); }
    __device__ __forceinline__ void wide(float (&f)[8]) const { Vec<T>::wide(v, f); }
    static __device__ __forceinline__ void store(T* p, const float (&f)[8]) { st16(p, Vec<T>::narrow(f)); }
};
template <> struct Eight<float> {
    float f[8];
    __device__ __forceinline__ void load(const float* p) {
        asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void wide(float (&g)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = f[i];
    }
    static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
        asm volatile("st.global.L1::no_allocate.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]) : "memory");
    }
};

// Whole blocks, one to a thread and access, NB of them under way per thread.  FLAT: rows without gaps are
// one row; else a row has `chunks` blocks.  DRAW: numbers are drawn, else all of them are 0.
template <typename T, bool RES, bool FLAT, bool DRAW, int NB, int TB>
__global__ void __launch_bounds__(TB) k_dropout(const DropoutArgs a, const int64_t blocks, const int64_t chunks) {
    const int64_t first = int64_t(blockIdx.x) * (NB * TB) + threadIdx.x;
    const Philox draw(a);
    auto some = [&](auto whole) {   // whole: every thread has NB blocks
        Eight<T> x[NB], res[RES ? NB : 1];
        int64_t at[NB] = {};   // the row
        auto element = [&](int i, int64_t ld) {
            const int64_t b = first + i * TB;
            return FLAT ? first * 8 + i * TB * 8 : at[i] * ld + (b - at[i] * chunks) * 8;
        };
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int64_t b = first + i * TB;
            if (!FLAT) at[i] = (b >> 32) == 0 && (chunks >> 32) == 0 ? int64_t(uint32_t(b) / uint32_t(chunks)) : b / chunks;
            if (decltype(whole)::value || b < blocks) {
                x[i].load(static_cast<const T*>(a.x) + element(i, a.ldx));
                if (RES) res[i].load(static_cast<const T*>(a.residual) + element(i, a.ldr));
            }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int64_t b = first + i * TB;
            if (!decltype(whole)::value && b >= blocks) break;
            const uint4 bits = DRAW ? draw(uint64_t(b)) : make_uint4(0, 0, 0, 0);
            float f[8], g[8];
            x[i].wide(f);
            if (RES) res[i].wide(g);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = dropped(f[j], kept(word_of(bits, j >> 1), j, a.limit), a.scale, RES ? g[j] : 0.0f);
            Eight<T>::store(static_cast<T*>(a.y) + element(i, a.ldy), f);
        }
    };
    if ((int64_t(blockIdx.x) + 1) * (NB * TB) <= blocks) some(std::true_type{}); else some(std::false_type{});
    // the elements behind the last whole block (of the one row)
    const int64_t n = blocks * 8 + threadIdx.x;
    if (FLAT && blockIdx.x == 0 && n < a.cols) {
        const uint4 bits = DRAW ? draw(uint64_t(blocks)) : make_uint4(0, 0, 0, 0);
        const float r = RES ? to_f(static_cast<const T*>(a.residual)[n]) : 0.0f;
        const bool keep = kept(word_of(bits, int(threadIdx.x) >> 1), int(threadIdx.x), a.limit);
        static_cast<T*>(a.y)[n] = from_f<T>(dropped(to_f(static_cast<const T*>(a.x)[n]), keep, a.scale, r));
    }
}

// Any strides and alignment, by elements: a warp draws 32 blocks, one per lane, and takes their 256
// elements in order, so that its accesses are of neighbouring elements.
template <typename T, bool RES, int TB>
__global__ void __launch_bounds__(TB) k_dropout_any(const DropoutArgs a, const int64_t numel) {
    __shared__ uint4 bits[TB];
    const Philox draw(a);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = (int64_t(blockIdx.x) * (TB / 32) + warp) * 256;
    if (first >= numel) return;
    T x[8], res[RES ? 8 : 1];
    int64_t to[8];   // the element's place in y
    int64_t row = a.rows == 1 ? 0 : (first + lane) / a.cols, col = first + lane - row * a.cols;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (first + 32 * i + lane < numel) {
            x[i] = static_cast<const T*>(a.x)[row * a.ldx + col];
            if (RES) res[i] = static_cast<const T*>(a.residual)[row * a.ldr + col];
        }
        to[i] = row * a.ldy + col;
        col += 32;
        if (a.cols >= 32) {
            if (col >= a.cols) {
                col -= a.cols;
                ++row;
            }
        } else {
            const int steps = int(col) / int(a.cols);
            row += steps;
            col -= steps * a.cols;
        }
    }
    bits[threadIdx.x] = a.random ? draw(uint64_t(first >> 3) + lane) : make_uint4(0, 0, 0, 0);
    __syncwarp();
    const uint32_t* const words = reinterpret_cast<const uint32_t*>(bits + warp * 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (first + 32 * i + lane >= numel) break;
        const bool keep = kept(words[(32 * i + lane) >> 1], lane, a.limit);
        static_cast<T*>(a.y)[to[i]] = from_f<T>(dropped(to_f(x[i]), keep, a.scale, RES ? to_f(res[i]) : 0.0f));
    }
}

// 16-bit rows whose vectors begin anywhere in a block, at one phase in all operands: a warp takes 128 vectors of a
// row in order, a lane draws the block that its vector begins in, and the numbers behind that block's end are the
// next lane's.  16,384 x 8,192 bf16 at an odd stride: 116 us; by elements 291.
template <typename T, bool RES, int TB>
__global__ void __launch_bounds__(TB) k_dropout_rows(const DropoutArgs a, const uint32_t segs) {
    static_assert(sizeof(T) == 2, "eight elements to a vector");
    constexpr int NB = 4;
    const Philox draw(a);
    const int lane = threadIdx.x & 31;
    const int64_t item = int64_t(blockIdx.x) * (TB / 32) + (threadIdx.x >> 5);
    const int64_t row = item >> 32 ? item / segs : int64_t(uint32_t(item) / segs);
    if (row >= a.rows) return;
    const int64_t v0 = (item - row * segs) * (32 * NB);
    const T* const x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* const res = RES ? static_cast<const T*>(a.residual) + row * a.ldr : nullptr;
    T* const y = static_cast<T*>(a.y) + row * a.ldy;
    const int64_t head = min(int64_t((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / 2, a.cols), body = (a.cols - head) / 8;
    Eight<T> in[NB], add[RES ? NB : 1];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int64_t v = v0 + 32 * i + lane;
        if (v < body) {
            in[i].load(x + head + v * 8);
            if (RES) add[i].load(res + head + v * 8);
        }
    }
    const int64_t e0 = row * a.cols + head + v0 * 8;
    const uint64_t q0 = uint64_t(e0 >> 3);
    const int shift = int(e0 & 7);
    uint4 own = draw(q0 + lane);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const uint4 next = draw(q0 + 32 * (i + 1) + lane);   // of the next 32 vectors
        uint32_t w[8] = {own.x, own.y, own.z, own.w, 0, 0, 0, 0};
        if (shift != 0) {   // the same for a whole row
            const int from = (lane + 1) & 31;
            w[4] = __shfl_sync(~0u, lane == 0 ? next.x : own.x, from);
            w[5] = __shfl_sync(~0u, lane == 0 ? next.y : own.y, from);
            w[6] = __shfl_sync(~0u, lane == 0 ? next.z : own.z, from);
            w[7] = __shfl_sync(~0u, lane == 0 ? next.w : own.w, from);
            if (shift & 4) {
#pragma unroll
                for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
            }
            if (shift & 2) {
#pragma unroll
                for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
            }
            if (shift & 1) {
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
            }
        }
        own = next;
        const int64_t v = v0 + 32 * i + lane;
        if (v >= body) continue;
        float f[8], g[8];
        in[i].wide(f);
        if (RES) add[i].wide(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = dropped(f[j], kept(w[j >> 1], j, a.limit), a.scale, RES ? g[j] : 0.0f);
        Eight<T>::store(y + head + v * 8, f);
    }
    // the row's first and last elements
    const int64_t c = lane < head ? lane : lane + body * 8;
    if (v0 == 0 && c < a.cols) {
        const int64_t e = row * a.cols + c;
        const bool keep = kept(word_of(draw(uint64_t(e >> 3)), int(e & 7) >> 1), int(e & 7), a.limit);
        y[c] = from_f<T>(dropped(to_f(x[c]), keep, a.scale, RES ? to_f(res[c]) : 0.0f));
    }
}

// From this many columns on: 16.8M bf16 elements at an odd stride take 59 / 40 / 29 / 19 us by rows of 257 / 400 / 600 / 1,001
// columns, 38 by elements from 129 to 400.
constexpr int64_t kRowColumns = 512;

template <typename T, bool RES>
cudaError_t launch(DropoutArgs a, cudaStream_t s) {
    constexpr int NB = kBlocks<RES>, TB = kDropThreads;
    const int64_t numel = a.rows * a.cols;
    if (a.rows > 1 && a.ldx == a.cols && a.ldy == a.cols && (!RES || a.ldr == a.cols)) {   // no gaps
        a.rows = 1;
        a.cols = a.ldx = a.ldr = a.ldy = numel;
    }
    constexpr uintptr_t unit = 8 * sizeof(T);
    bool whole = aligned(a.x, unit) && aligned(a.y, unit) && (!RES || aligned(a.residual, unit));
    if (a.rows > 1) whole = whole && a.cols % 8 == 0 && a.ldx % 8 == 0 && a.ldy % 8 == 0 && (!RES || a.ldr % 8 == 0);
    if constexpr (sizeof(T) == 2) {
        auto phase = [&](const void* p) { return ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(a.x)) & 15) == 0; };
        const bool alike = phase(a.y) && (!RES || phase(a.residual)) &&
                           (a.rows == 1 || ((a.ldx - a.ldy) % 8 == 0 && (!RES || (a.ldx - a.ldr) % 8 == 0)));
        if (!whole && a.random && alike && a.cols >= kRowColumns && a.cols < (int64_t(1) << 38)) {
            const int64_t segs = (a.cols / 8 + 127) / 128, warps = a.rows * segs, need = (warps + TB / 32 - 1) / (TB / 32);
            if (need <= 0x7fffffff) {
                k_dropout_rows<T, RES, TB><<<unsigned(need), TB, 0, s>>>(a, uint32_t(segs));
                return cudaGetLastError();
            }
        }
    }
    const int64_t per = whole ? int64_t(NB) * TB * 8 : int64_t(TB) * 8, ctas = (numel + per - 1) / per;
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    if (whole && a.rows == 1) {
        auto* kernel = a.random ? k_dropout<T, RES, true, true, NB, TB> : k_dropout<T, RES, true, false, NB, TB>;
        kernel<<<unsigned(ctas), TB, 0, s>>>(a, numel / 8, 0);
    } else if (whole) {
        auto* kernel = a.random ? k_dropout<T, RES, false, true, NB, TB> : k_dropout<T, RES, false, false, NB, TB>;
        kernel<<<unsigned(ctas), TB, 0, s>>>(a, numel / 8, a.cols / 8);
    } else
        k_dropout_any<T, RES, TB><<<unsigned(ctas), TB, 0, s>>>(a, numel);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_by(const DropoutArgs& a, cudaStream_t s) {
    return a.residual ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

// The last error of the calling thread: a call has no context that would hold it.
thread_local const char* last_error = "";
int fail(int code, const char* text) {
    last_error = text;
    return code;
}

// One matrix operand: its address and stride.
bool operand(const void* p, int64_t ld, int64_t rows, int64_t cols, int64_t size) {
    return p != nullptr && aligned(p, uintptr_t(size)) && ld >= cols && (rows == 1 || (ld < kMaxLd && ld <= kMaxSpan / rows));
}

}  // namespace
}  // namespace tl

using namespace tl;

extern "C" const char* tl_dropout_last_error(void) { return last_error; }

extern "C" int tl_dropout(const tl_dropout_args* args, tl_stream stream) {
    if (args == nullptr) return fail(TL_EINVAL, "args must not be NULL");
    const tl_dropout_args& g = *args;
    if (!float_type(g.dtype)) return fail(TL_EINVAL, "dtype must be TL_F32, TL_BF16 or TL_F16");
    if (!(g.p >= 0.0f && g.p <= 1.0f)) return fail(TL_EINVAL, "p must be in [0, 1]");
    if (g.rows < 0 || g.cols < 0 || too_many(g.rows, g.cols))
        return fail(TL_EINVAL, "rows and cols must be at least 0, rows * cols at most 2^40");
    if (g.key == nullptr || !aligned(g.key, 8)) return fail(TL_EINVAL, "key must be an address aligned to 8 bytes");
    const int64_t size = type_bytes(g.dtype);
    if (g.rows > 0 && g.cols > 0) {
        if (!operand(g.x, g.ldx, g.rows, g.cols, size)) return fail(TL_EINVAL, "x must be an aligned address, ldx in [cols, 2^40)");
        if (!operand(g.y, g.ldy, g.rows, g.cols, size)) return fail(TL_EINVAL, "y must be an aligned address, ldy in [cols, 2^40)");
        if (g.residual != nullptr && !operand(g.residual, g.ldr, g.rows, g.cols, size))
            return fail(TL_EINVAL, "residual must be an aligned address, ldr in [cols, 2^40)");
        if (rows_clash(g.x, g.ldx, g.y, g.ldy, g.rows, g.cols, size))
            return fail(TL_EINVAL, "y overlaps x without being the same tensor");
        if (g.residual != nullptr && rows_clash(g.residual, g.ldr, g.y, g.ldy, g.rows, g.cols, size))
            return fail(TL_EINVAL, "y overlaps residual without being the same tensor");
        Spans sp;
        sp.add(g.key, 16, false);
        sp.add(g.y, span_bytes(g.rows, g.cols, g.ldy, size), true);
        if (sp.clash()) return fail(TL_EINVAL, "y overlaps key");
    }
    int dev = -1;
    const cudaError_t asked = cudaGetDevice(&dev);
    if (asked != cudaSuccess) return fail(TL_ECUDA, cudaGetErrorString(asked));
    if (dev != g.device) return fail(TL_ESTATE, "the current CUDA device is not the tensors' device");
    if (g.rows == 0 || g.cols == 0) return TL_OK;
    const uint32_t P = uint32_t(std::lrint(double(g.p) * 65536.0));
    DropoutArgs a{};
    a.x = g.x;
    a.residual = g.residual;
    a.y = g.y;
    a.rows = g.rows;
    a.cols = g.cols;
    a.ldx = g.ldx;
    a.ldr = g.ldr;
    a.ldy = g.ldy;
    a.key = g.key;
    a.site = g.site;
    // where all or none are kept nothing is drawn: 0 is kept, or below the limit
    a.random = P > 0 && P < 65536;
    a.limit = P < 65536 ? P << 16 : 1u;
    a.scale = P < 65536 ? float(65536.0 / (65536.0 - double(P))) : 0.0f;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = g.dtype == TL_F32 ? launch_by<float>(a, s)
                          : g.dtype == TL_BF16 ? launch_by<__nv_bfloat16>(a, s) : launch_by<__half>(a, s);
    return e == cudaSuccess ? TL_OK : fail(TL_ECUDA, cudaGetErrorString(e));
}
