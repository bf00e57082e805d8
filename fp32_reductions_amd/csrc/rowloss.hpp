// rowloss.hpp -- host-side interface between the C ABI (api.hip) and the
// kernels of the losses over rows of logits (rowloss_kernels.hpp,
// instantiated per element type in rowloss_f32.hip, rowloss_f16.hip and
// rowloss_bf16.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.hpp"

namespace red {

// Element types of logits and their gradients.
enum class LogitType { F32, F16, BF16 };

// Rows one launch covers.  A launch holds at most 2^32 - 1 work-items and a
// row takes at most 1024 of a launch that keeps rows whole (those that cut rows
// up have their own bounds), and the row losses of a launch (8 bytes each) fill
// at most half of the workspace; more rows take several launches.
constexpr size_t kRowsPerLaunch = size_t(1) << 20;
// Rows and pairs of a preference loss, whose per-row statistics (20 bytes a
// row) and pair losses (8 bytes) all stay in the workspace.
constexpr size_t kPrefRowsMax = size_t(1) << 19;
constexpr size_t kPrefPairsMax = size_t(1) << 17;
// Teacher entries per row, and columns of a distilled row: the entries (12
// bytes each) and a bit per column stay in at most 64 KiB of LDS.
constexpr size_t kTopkMax = 1024;
constexpr size_t kTopkColsMax = 393216;

// A row-major matrix of logits and, where dz is not null, of its gradient.
struct Logits {
    const void* z;
    void* dz;
    size_t rows, V, ld, ldd;
    float scale;
};

struct LogprobCall {
    Logits m;
    const int64_t* targets;
    float *logp, *lse, *entropy;
};

struct LogprobGradCall {
    Logits m;
    const int64_t* targets;
    const float *lse, *entropy, *glogp, *gentropy;
};

struct DistillCall {
    Logits m;
    const int64_t* idx;
    const float* val;
    size_t K, ldk;
    const float *teacher_lse, *weight;
    float *loss, *row_loss;
    int accum;
};

struct PolicyCall {
    Logits m;
    const int64_t* targets;
    const float *old_logp, *ref_logp, *advantage, *weight;
    float clip_low, clip_high, kl_coef, entropy_coef;
    float *loss, *logp, *entropy;
    int accum;
};

struct PreferenceCall {
    Logits m;
    const int64_t* targets;
    const int64_t* starts;
    size_t pairs;
    const float *ref_logp, *weight;
    int kind, average;
    float beta, margin, smoothing;
    float *loss, *seq_logp;
    int accum;
};

// Whether the call keeps something in the workspace.
bool token_logprob_shares(LogitType t, const Logits& m);
hipError_t launch_token_logprob(LogitType t, const LogprobCall& a, const DeviceInfo& dev,
                                const Workspace& ws, hipStream_t stream);
hipError_t launch_token_logprob_grad(LogitType t, const LogprobGradCall& a,
                                     const DeviceInfo& dev, hipStream_t stream);
hipError_t launch_distill_topk(LogitType t, const DistillCall& a, const DeviceInfo& dev,
                               const Workspace& ws, hipStream_t stream);
hipError_t launch_policy_loss(LogitType t, const PolicyCall& a, const DeviceInfo& dev,
                              const Workspace& ws, hipStream_t stream);
hipError_t launch_preference_loss(LogitType t, const PreferenceCall& a, const DeviceInfo& dev,
                                  const Workspace& ws, hipStream_t stream);

// The kernels of one element type (T: a trait of rowloss_kernels.hpp).
template <class T>
struct RowLoss {
    static bool logprob_shares(const Logits& m);
    static hipError_t logprob(const LogprobCall& a, const DeviceInfo& dev, const Workspace& ws,
                              hipStream_t stream);
    static hipError_t logprob_grad(const LogprobGradCall& a, const DeviceInfo& dev,
                                   hipStream_t stream);
    static hipError_t distill(const DistillCall& a, const DeviceInfo& dev, const Workspace& ws,
                              hipStream_t stream);
    static hipError_t policy(const PolicyCall& a, const DeviceInfo& dev, const Workspace& ws,
                             hipStream_t stream);
    static hipError_t preference(const PreferenceCall& a, const DeviceInfo& dev,
                                 const Workspace& ws, hipStream_t stream);
};
struct ElemF32;
struct ElemF16;
struct ElemBF16;
extern template struct RowLoss<ElemF32>;
extern template struct RowLoss<ElemF16>;
extern template struct RowLoss<ElemBF16>;

// loss[0] = [loss[0] +] sum of n row losses (rowloss.hip).  `before` (null: 0)
// is added in fp64; where `after` is not null the sum goes there, and not to
// loss: of several launches that make one loss only the last rounds it.
hipError_t launch_loss_sum(const double* row_loss, size_t n, float* loss, int accum,
                           const double* before, double* after, hipStream_t stream);
} // namespace red
