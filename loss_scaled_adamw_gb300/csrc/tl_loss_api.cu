// tl_loss_api.cu - host side of the objectives declared in include/tl_loss.h: the
// context (scratch for row statistics and sums), the checks of every argument
// before any launch, and the launches.
#include "tl_loss_internal.cuh"

#include <cfloat>
#include <cmath>
#include <new>
#include <string>

#include "../../include/tl_loss.h"

using namespace tl;

struct tl_loss_ctx {
    int device = 0;
    int sm_count = 0;
    int64_t max_rows = 0;
    int64_t max_pairs = 0;
    RowStat* d_stat = nullptr;     // preference: one per row
    double* d_slots = nullptr;     // 4 sums per row group of a launch
    uint32_t* d_ticket = nullptr;  // row groups that have finished; zero between calls
    GroupCache cache;
    int64_t launches = 0;
    std::string last_error;
};

namespace {

// Nothing is thrown across the C boundary: a message that cannot be stored is dropped.
int fail(tl_loss_ctx* ctx, int code, const char* msg, const char* detail = nullptr) noexcept {
    try {
        ctx->last_error = msg;
        if (detail) ctx->last_error.append(": ").append(detail);
    } catch (...) {
        ctx->last_error.clear();
    }
    return code;
}

int cuda_fail(tl_loss_ctx* ctx, cudaError_t e, const char* what) noexcept {
    return fail(ctx, TL_ECUDA, what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool float_type(int dt) { return dt == TL_F32 || dt == TL_BF16 || dt == TL_F16; }
int64_t type_bytes(int dt) { return dt == TL_F32 ? 4 : 2; }
bool weight(float v) { return v >= 0.0f && std::isfinite(v); }

// Element offsets stay far from 2^63: rows < 2^31, ld < 2^40 would reach 2^71, so
// the product is bounded too.
constexpr int64_t kMaxLd = int64_t(1) << 40;
constexpr int64_t kMaxSpan = int64_t(1) << 56;

// The memory a call touches: no output may share bytes with anything else.
struct Spans {
    struct One {
        uintptr_t lo, hi;
        bool out;
    } v[16];
    int n = 0;
    void add(const void* p, int64_t bytes, bool out) {
        if (p == nullptr || bytes <= 0) return;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        v[n++] = {lo, lo + uintptr_t(bytes), out};
    }
    bool clash() const {
        for (int i = 0; i < n; ++i)
            for (int j = i + 1; j < n; ++j)
                if ((v[i].out || v[j].out) && v[i].lo < v[j].hi && v[j].lo < v[i].hi) return true;
        return false;
    }
};

int64_t span_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t size) {
    return rows < 1 || cols < 1 ? 0 : ((rows - 1) * ld + cols) * size;
}

// Whether two row-strided matrices of one shape share an element: equal strides
// interleave when their columns stay apart, others are held to disjoint spans.
bool rows_clash(const tl_logits& x, const void* d, int64_t ldd) {
    const int64_t size = type_bytes(x.dtype);
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.data), b = reinterpret_cast<uintptr_t>(d);
    const uintptr_t ahi = a + uintptr_t(span_bytes(x.rows, x.vocab, x.ld, size));
    const uintptr_t bhi = b + uintptr_t(span_bytes(x.rows, x.vocab, ldd, size));
    if (a >= bhi || b >= ahi) return false;
    if (x.ld != ldd) return true;
    if (a == b) return false;   // in place
    const uintptr_t stride = uintptr_t(x.ld * size), width = uintptr_t(x.vocab * size);
    const uintptr_t off = (a < b ? b - a : a - b) % stride;
    return off < width || off + width > stride;
}

int check_device(tl_loss_ctx* ctx) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(ctx, e, "cudaGetDevice");
    if (dev != ctx->device) return fail(ctx, TL_ESTATE, "the current CUDA device is not the context's device");
    return TL_OK;
}

int check_logits(tl_loss_ctx* ctx, const tl_logits* x) {
    if (x == nullptr) return fail(ctx, TL_EINVAL, "logits must not be NULL");
    if (!float_type(x->dtype)) return fail(ctx, TL_EINVAL, "logits dtype must be TL_F32, TL_BF16 or TL_F16");
    if (x->rows < 0 || x->rows > ctx->max_rows) return fail(ctx, TL_EINVAL, "rows must be in [0, max_rows]");
    if (x->vocab < 1 || x->vocab > (int64_t(1) << 30)) return fail(ctx, TL_EINVAL, "vocab must be in [1, 2^30]");
    if (x->ld < x->vocab || x->ld >= kMaxLd) return fail(ctx, TL_EINVAL, "ld must be in [vocab, 2^40)");
    if (x->rows > 0 && x->ld > kMaxSpan / x->rows) return fail(ctx, TL_EINVAL, "rows * ld must be at most 2^56");
    if (!(x->temperature >= FLT_MIN) || !std::isfinite(x->temperature) || !std::isnormal(1.0f / x->temperature))
        return fail(ctx, TL_EINVAL, "temperature must be positive, normal and have a normal reciprocal");
    if (x->rows > 0 && (x->data == nullptr || !aligned(x->data, uintptr_t(type_bytes(x->dtype)))))
        return fail(ctx, TL_EINVAL, "logits must be an address aligned to their element size");
    return TL_OK;
}

// Fills the parts of the launch arguments that every call shares.
void base_args(tl_loss_ctx* ctx, const tl_logits* x, const int64_t* target, LossArgs& a, Spans& sp) {
    a = LossArgs{};
    a.x = x->data;
    a.ld = x->ld;
    a.rows = x->rows;
    a.vocab = int32_t(x->vocab);
    a.it = 1.0f / x->temperature;
    a.target = target;
    a.stat = ctx->d_stat;
    a.slots = ctx->d_slots;
    a.ticket = ctx->d_ticket;
    a.inv_n = 1.0f;
    a.per_n = 1.0;
    sp.add(target, 8 * x->rows, false);
}

int check_floats(tl_loss_ctx* ctx, const void* p, bool required, const char* name) {
    if (p == nullptr ? required : !aligned(p, 4)) return fail(ctx, TL_EINVAL, name, "missing or misaligned");
    return TL_OK;
}

int check_target(tl_loss_ctx* ctx, const tl_logits* x, const int64_t* target, bool required) {
    if (target == nullptr ? required && x->rows > 0 : !aligned(target, 8))
        return fail(ctx, TL_EINVAL, "target", "missing or misaligned");
    return TL_OK;
}

// The outputs of a loss call; `losses`: how many floats out->loss holds.
int check_out(tl_loss_ctx* ctx, const tl_logits* x, const tl_loss_out* o, int64_t losses, LossArgs& a, Spans& sp) {
    if (o == nullptr) return fail(ctx, TL_EINVAL, "out must not be NULL");
    if (o->n < 1 || o->n > (int64_t(1) << 53)) return fail(ctx, TL_EINVAL, "n must be in [1, 2^53]");
    int rc;
    if ((rc = check_floats(ctx, o->seed, false, "seed")) != TL_OK) return rc;
    if ((rc = check_floats(ctx, o->logp, false, "logp")) != TL_OK) return rc;
    if ((rc = check_floats(ctx, o->loss, false, "loss")) != TL_OK) return rc;
    if ((rc = check_floats(ctx, o->result, true, "result")) != TL_OK) return rc;
    if (o->dlogits != nullptr) {
        if (!aligned(o->dlogits, uintptr_t(type_bytes(x->dtype))))
            return fail(ctx, TL_EINVAL, "dlogits must be aligned to their element size");
        if (o->ld_dlogits < x->vocab || o->ld_dlogits >= kMaxLd)
            return fail(ctx, TL_EINVAL, "ld_dlogits must be in [vocab, 2^40)");
        if (x->rows > 0 && o->ld_dlogits > kMaxSpan / x->rows)
            return fail(ctx, TL_EINVAL, "rows * ld_dlogits must be at most 2^56");
        if (rows_clash(*x, o->dlogits, o->ld_dlogits))
            return fail(ctx, TL_EINVAL, "dlogits overlap the logits without being the same tensor");
    }
    a.dx = o->dlogits;
    a.ldd = o->ld_dlogits;
    a.seed = o->seed;
    a.inv_n = float(1.0 / double(o->n));
    a.per_n = 1.0 / double(o->n);
    a.logp = o->logp;
    a.loss = o->loss;
    a.result = reinterpret_cast<float*>(o->result);
    sp.add(o->seed, 4, false);
    sp.add(o->logp, 4 * x->rows, true);
    sp.add(o->loss, 4 * losses, true);
    sp.add(o->result, 16, true);
    return TL_OK;
}

// No output shares memory with anything else (the logits / dlogits pair apart,
// which rows_clash has looked at).
int check_spans(tl_loss_ctx* ctx, const tl_logits* x, const LossArgs& a, const Spans& sp) {
    Spans with_x = sp, with_dx = sp;
    with_x.add(x->data, span_bytes(x->rows, x->vocab, x->ld, type_bytes(x->dtype)), false);
    if (a.dx) with_dx.add(a.dx, span_bytes(x->rows, x->vocab, a.ldd, type_bytes(x->dtype)), true);
    if (with_x.clash() || with_dx.clash()) return fail(ctx, TL_EINVAL, "an output overlaps another argument");
    return check_device(ctx);
}

int run_rows(tl_loss_ctx* ctx, int op, int dt, const LossArgs& a, tl_stream stream) {
    cudaError_t e = launch_loss_rows(op, dt, a, ctx->sm_count, ctx->cache, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(ctx, e, "objective launch");
    ctx->launches += 1;
    return TL_OK;
}

void free_ctx(tl_loss_ctx* ctx) {
    cudaFree(ctx->d_stat);
    cudaFree(ctx->d_slots);
    cudaFree(ctx->d_ticket);
    delete ctx;
}

}  // namespace

extern "C" {

int tl_loss_create(tl_loss_ctx** out, int64_t max_rows, int64_t max_pairs, tl_stream stream) {
    if (out == nullptr) return TL_EINVAL;
    *out = nullptr;
    if (max_rows < 0 || max_rows > (int64_t(1) << 31) - 1 || max_pairs < 0 || max_pairs > (int64_t(1) << 28))
        return TL_EINVAL;
    tl_loss_ctx* ctx = new (std::nothrow) tl_loss_ctx();
    if (ctx == nullptr) return TL_ENOMEM;
    ctx->max_rows = max_rows;
    ctx->max_pairs = max_pairs;
    cudaError_t e = cudaGetDevice(&ctx->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&ctx->sm_count, cudaDevAttrMultiProcessorCount, ctx->device);
    if (e != cudaSuccess) { free_ctx(ctx); return TL_ECUDA; }
    const int64_t stats = max_pairs > 0 ? max_rows : 0;
    if (cudaMalloc(&ctx->d_stat, sizeof(RowStat) * size_t(stats < 1 ? 1 : stats)) != cudaSuccess ||
        cudaMalloc(&ctx->d_slots, sizeof(double) * 4 * kMaxLossClusters) != cudaSuccess ||
        cudaMalloc(&ctx->d_ticket, sizeof(uint32_t)) != cudaSuccess) {
        cudaGetLastError();
        free_ctx(ctx);
        return TL_ENOMEM;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    e = cudaMemsetAsync(ctx->d_ticket, 0, sizeof(uint32_t), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) { free_ctx(ctx); return TL_ECUDA; }
    *out = ctx;
    return TL_OK;
}

int tl_loss_destroy(tl_loss_ctx* ctx) {
    if (ctx == nullptr) return TL_OK;
    cudaError_t e = cudaDeviceSynchronize();
    free_ctx(ctx);
    return e == cudaSuccess ? TL_OK : TL_ECUDA;
}

int tl_token_logprob(tl_loss_ctx* ctx, const tl_logits* logits, const int64_t* target, float* logp,
                     tl_stream stream) {
    if (ctx == nullptr) return TL_EINVAL;
    int rc;
    LossArgs a;
    Spans sp;
    if ((rc = check_logits(ctx, logits)) != TL_OK) return rc;
    if ((rc = check_target(ctx, logits, target, true)) != TL_OK) return rc;
    if ((rc = check_floats(ctx, logp, logits->rows > 0, "logp")) != TL_OK) return rc;
    base_args(ctx, logits, target, a, sp);
    a.logp = logp;
    sp.add(logp, 4 * logits->rows, true);
    if ((rc = check_spans(ctx, logits, a, sp)) != TL_OK) return rc;
    if (logits->rows == 0) return TL_OK;
    return run_rows(ctx, kLogprob, logits->dtype, a, stream);
}

int tl_policy_loss(tl_loss_ctx* ctx, const tl_logits* logits, const tl_policy_args* args, const tl_loss_out* out,
                   tl_stream stream) {
    if (ctx == nullptr) return TL_EINVAL;
    int rc;
    LossArgs a;
    Spans sp;
    if ((rc = check_logits(ctx, logits)) != TL_OK) return rc;
    if (args == nullptr) return fail(ctx, TL_EINVAL, "args must not be NULL");
    const bool some = logits->rows > 0;
    if ((rc = check_target(ctx, logits, args->target, true)) != TL_OK) return rc;
    if ((rc = check_floats(ctx, args->old_logp, some, "old_logp")) != TL_OK) return rc;
    if ((rc = check_floats(ctx, args->advantage, some, "advantage")) != TL_OK) return rc;
    if ((rc = check_floats(ctx, args->ref_logp, false, "ref_logp")) != TL_OK) return rc;
    if (!weight(args->clip_low) || args->clip_low > 1.0f || !weight(args->clip_high) ||
        !std::isfinite(1.0f + args->clip_high))
        return fail(ctx, TL_EINVAL, "clip_low must be in [0, 1] and clip_high >= 0");
    if (!weight(args->kl_weight)) return fail(ctx, TL_EINVAL, "kl_weight must be finite and >= 0");
    if (args->kl_weight > 0.0f && args->ref_logp == nullptr && some)
        return fail(ctx, TL_EINVAL, "kl_weight > 0 needs ref_logp");
    base_args(ctx, logits, args->target, a, sp);
    if ((rc = check_out(ctx, logits, out, logits->rows, a, sp)) != TL_OK) return rc;
    a.old_logp = args->old_logp;
    a.ref_logp = args->ref_logp;
    a.adv = args->advantage;
    a.lo = 1.0f - args->clip_low;
    a.hi = 1.0f + args->clip_high;
    a.kl_weight = args->kl_weight;
    sp.add(a.old_logp, 4 * a.rows, false);
    sp.add(a.ref_logp, 4 * a.rows, false);
    sp.add(a.adv, 4 * a.rows, false);
    if ((rc = check_spans(ctx, logits, a, sp)) != TL_OK) return rc;
    return run_rows(ctx, kPolicy, logits->dtype, a, stream);
}

int tl_preference_loss(tl_loss_ctx* ctx, const tl_logits* logits, const tl_preference_args* args,
                       const tl_loss_out* out, tl_stream stream) {
    if (ctx == nullptr) return TL_EINVAL;
    int rc;
    LossArgs a;
    Spans sp;
    if ((rc = check_logits(ctx, logits)) != TL_OK) return rc;
    if (args == nullptr) return fail(ctx, TL_EINVAL, "args must not be NULL");
    if ((rc = check_target(ctx, logits, args->target, true)) != TL_OK) return rc;
    if (args->pairs < 0 || args->pairs > ctx->max_pairs) return fail(ctx, TL_EINVAL, "pairs must be in [0, max_pairs]");
    if (ctx->max_pairs == 0) return fail(ctx, TL_EINVAL, "the context was created without preference pairs");
    if (args->seq == nullptr ? args->pairs > 0 : !aligned(args->seq, 8))
        return fail(ctx, TL_EINVAL, "seq", "missing or misaligned");
    if ((rc = check_floats(ctx, args->ref_logp, false, "ref_logp")) != TL_OK) return rc;
    if ((rc = check_floats(ctx, args->reward, false, "reward")) != TL_OK) return rc;
    if (!weight(args->beta) || args->beta == 0.0f) return fail(ctx, TL_EINVAL, "beta must be positive and finite");
    if (!weight(args->label_smoothing) || args->label_smoothing > 0.5f)
        return fail(ctx, TL_EINVAL, "label_smoothing must be in [0, 0.5]");
    base_args(ctx, logits, args->target, a, sp);
    if ((rc = check_out(ctx, logits, out, args->pairs, a, sp)) != TL_OK) return rc;
    a.seq = args->seq;
    a.pairs = args->pairs;
    a.ref_logp = args->ref_logp;
    a.beta = args->beta;
    a.smooth = args->label_smoothing;
    a.reward = args->reward;
    sp.add(a.seq, 8 * (2 * a.pairs + 1), false);
    sp.add(a.ref_logp, 4 * a.rows, false);
    sp.add(a.reward, 8 * a.pairs, true);
    if ((rc = check_spans(ctx, logits, a, sp)) != TL_OK) return rc;
    if ((rc = run_rows(ctx, kPrefStat, logits->dtype, a, stream)) != TL_OK) return rc;
    if (a.dx == nullptr || a.rows == 0) return TL_OK;
    cudaError_t e = launch_pref_grad(logits->dtype, a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(ctx, e, "preference gradient launch");
    ctx->launches += 1;
    return TL_OK;
}

int tl_distill_loss(tl_loss_ctx* ctx, const tl_logits* logits, const tl_distill_args* args, const tl_loss_out* out,
                    tl_stream stream) {
    if (ctx == nullptr) return TL_EINVAL;
    int rc;
    LossArgs a;
    Spans sp;
    if ((rc = check_logits(ctx, logits)) != TL_OK) return rc;
    if (args == nullptr) return fail(ctx, TL_EINVAL, "args must not be NULL");
    if (!weight(args->kd_weight) || !weight(args->ce_weight))
        return fail(ctx, TL_EINVAL, "kd_weight and ce_weight must be finite and >= 0");
    if ((rc = check_target(ctx, logits, args->target, args->ce_weight > 0.0f)) != TL_OK) return rc;
    if (args->k < 0 || args->k > kMaxTeacher) return fail(ctx, TL_EINVAL, "k must be in [0, 1024]");
    if (args->k > 0) {
        if (!float_type(args->teacher_dtype)) return fail(ctx, TL_EINVAL, "teacher_dtype must be TL_F32, TL_BF16 or TL_F16");
        if (args->id_bytes != 4 && args->id_bytes != 8) return fail(ctx, TL_EINVAL, "id_bytes must be 4 or 8");
        if (args->ld_teacher < args->k || args->ld_teacher >= kMaxLd ||
            (logits->rows > 0 && args->ld_teacher > kMaxSpan / logits->rows))
            return fail(ctx, TL_EINVAL, "ld_teacher must be in [k, 2^40), rows * ld_teacher at most 2^56");
        if (logits->rows > 0 &&
            (args->teacher == nullptr || !aligned(args->teacher, uintptr_t(type_bytes(args->teacher_dtype))) ||
             args->teacher_id == nullptr || !aligned(args->teacher_id, uintptr_t(args->id_bytes))))
            return fail(ctx, TL_EINVAL, "teacher and teacher_id must be addresses aligned to their element size");
    }
    base_args(ctx, logits, args->target, a, sp);
    if ((rc = check_out(ctx, logits, out, logits->rows, a, sp)) != TL_OK) return rc;
    if (out->logp != nullptr) return fail(ctx, TL_EINVAL, "logp is not an output of the distillation loss");
    a.kd_weight = args->kd_weight;
    a.ce_weight = args->ce_weight;
    a.k = args->kd_weight > 0.0f ? args->k : 0;   // without weight the teacher is not read
    if (a.k == 0) {
        a.it = 1.0f;   // the cross-entropy alone is at temperature 1
    } else {
        a.teacher = args->teacher;
        a.tid = args->teacher_id;
        a.ldt = args->ld_teacher;
        a.teacher_dtype = args->teacher_dtype;
        a.id_bytes = args->id_bytes;
        sp.add(a.teacher, span_bytes(a.rows, a.k, a.ldt, type_bytes(a.teacher_dtype)), false);
        sp.add(a.tid, span_bytes(a.rows, a.k, a.ldt, a.id_bytes), false);
    }
    if ((rc = check_spans(ctx, logits, a, sp)) != TL_OK) return rc;
    return run_rows(ctx, kDistill, logits->dtype, a, stream);
}

int64_t tl_loss_launch_count(const tl_loss_ctx* ctx) { return ctx == nullptr ? 0 : ctx->launches; }

const char* tl_loss_last_error(const tl_loss_ctx* ctx) { return ctx == nullptr ? "" : ctx->last_error.c_str(); }

}  // extern "C"
