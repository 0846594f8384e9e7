// tl_loss_internal.cuh - types shared by the kernels over logits (tl_loss_kernels.cu,
// tl_stats_kernels.cu) and their host side (tl_loss_api.cu).  Not installed; the public interface is
// include/tl_loss.h.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace tl {

// What a row kernel does with a row's softmax.
enum LossOp : int {
    kLogprob = 0,     // the target's log-probability
    kPolicy = 1,      // clipped policy objective, forward (and backward when dx is set)
    kPrefStat = 2,    // preference, first pass: row statistics and log-ratios, then the pairs
    kDistill = 3      // distillation, forward (and backward when dx is set)
};

constexpr int kMaxTeacher = 1024;      // teacher entries per row
constexpr int kMaxLossClusters = 4096; // partial slots of the loss sums: most row groups of a launch

// What the second preference pass needs of a row: its softmax and the factor of
// its gradient (0 for ignored rows).
struct RowStat {
    float m;      // largest logit
    float rs;     // 1 / sum of exp((x - m) / temperature)
    float w;      // d loss / d z of the target is w * (1 - q)
    float ratio;  // first pass: lp - ref_logp
};

struct LossArgs {
    const void* x;
    int64_t ld;
    int64_t rows;
    int32_t vocab;
    float it;              // 1 / temperature
    const int64_t* target; // null: every row is valid (distill)
    // gradient
    void* dx;
    int64_t ldd;
    const float* seed;
    float inv_n;
    double per_n;          // 1 / n
    // policy
    const float* old_logp;
    const float* ref_logp;
    const float* adv;
    float lo, hi, kl_weight;
    // preference
    const int64_t* seq;
    int64_t pairs;
    float beta, smooth;
    float* reward;
    RowStat* stat;
    // distill
    const void* teacher;
    const void* tid;
    int64_t ldt;
    int32_t k;
    int32_t teacher_dtype;
    int32_t id_bytes;
    float kd_weight, ce_weight;
    // outputs
    float* logp;
    float* loss;
    float* result;
    // scratch: one slot of sums per row group, and the count of groups that finished
    double* slots;
    uint32_t* ticket;
};

constexpr int kMaxAlternatives = 256;  // alternatives per row

// tl_token_stats: a row's softmax statistics and its largest entries.
struct StatsArgs {
    const void* x;
    int64_t ld;
    int64_t rows;
    int32_t vocab;
    float it;              // 1 / temperature
    float c2, c2_low;      // log2 e / temperature, and what its rounding left out
    const int64_t* target; // null: every row is valid, no logp
    float* logp;
    float* entropy;
    float* saved;          // three per row: largest logit, log of the sum against it, entropy
    void* top_id;
    float* top_logp;
    int64_t ld_top;
    int32_t k;
    int32_t id_bytes;
};

// tl_token_grad: the gradient of log-probabilities and entropies.
struct TokenGradArgs {
    const void* x;
    int64_t ld;
    int64_t rows;
    int32_t vocab;
    float it, c2;          // as above
    const int64_t* target;
    const float* saved;
    const float* grad_logp;
    const float* grad_entropy;
    const float* seed;
    void* dx;
    int64_t ldd;
};

// Row groups that each kernel form can have resident at once on the context's device
// (asking the runtime for it costs more than a small launch).  A group waits for
// nothing outside itself, so this sizes the grid and no more.
struct GroupCache {
    static constexpr int kEntries = 128;
    struct Entry {
        const void* kernel;
        int threads, cluster, smem, groups;
    } v[kEntries];
    int n = 0;
};

// Launchers (tl_loss_kernels.cu).  dt: element type of the logits.
cudaError_t launch_loss_rows(int op, int dt, const LossArgs& a, int sm_count, GroupCache& cache, cudaStream_t s);
cudaError_t launch_pref_grad(int dt, const LossArgs& a, cudaStream_t s);

// Launchers (tl_stats_kernels.cu).
cudaError_t launch_token_stats(int dt, const StatsArgs& a, int sm_count, GroupCache& cache, cudaStream_t s);
cudaError_t launch_token_grad(int dt, const TokenGradArgs& a, cudaStream_t s);

}  // namespace tl
