// rowloss_pairs.hpp -- the pairs of a preference loss: from the rows'
// log-probabilities to the sequences', the pairs' losses and the rows' slopes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "reduce.h"
#include "rowloss.hpp"
#include "rowloss_join.hpp"

namespace red {

struct PairArgs {
    double* row_logp;
    float* row_slope;
    const int64_t *targets, *starts;
    const float *ref_logp, *weight;
    float* seq_logp;
    Join join;
    int64_t rows, V;
    uint32_t pairs;
    int kind, average;
    double beta, margin, smoothing;
    unsigned* counts; // of the rows of each pair
};

// What a pair loads besides its rows; early, so that nothing waits for it.
struct PairValues {
    double weight, ref[2];
    __device__ __forceinline__ PairValues(const PairArgs& a, uint32_t p)
    {
        // Without a branch: something else is read where there is no value.
        const float* some = reinterpret_cast<const float*>(a.starts);
        const float w = (a.weight ? a.weight : some)[p];
        const float r0 = (a.ref_logp ? a.ref_logp : some)[p];
        const float r1 = (a.ref_logp ? a.ref_logp : some)[(uint64_t)a.pairs + p];
        weight = a.weight ? (double)w : 1.0 / (double)a.pairs;
        ref[0] = a.ref_logp ? (double)r0 : 0.0;
        ref[1] = a.ref_logp ? (double)r1 : 0.0;
    }
};

// A pair from the sums of its sequences' log-probabilities and the counts of
// their rows: [0] chosen, [1] rejected.
struct PairResult {
    double seq[2], loss; // loss: with the pair's weight
    float slope[2];      // of the loss to a row's log-probability
    __device__ __forceinline__ PairResult(const PairArgs& a, const PairValues& v,
                                          const double (&sum)[2], const double (&count)[2])
    {
        double rows[2];
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            rows[side] = a.average && count[side] > 0.0 ? count[side] : 1.0;
            seq[side] = sum[side] / rows[side];
        }
        const double w = v.weight, delta = (seq[0] - v.ref[0]) - (seq[1] - v.ref[1]);
        const double h = a.beta * delta - a.margin;
        double l, dl; // the loss and its derivative to h
        if (a.kind == RED_PREF_SIGMOID) {
            // softplus(x) = max(x, 0) + log1p(exp(-|x|))
            const double t = exp(-fabs(h)), ln = log1p(t);
            const double pos = fmax(h, 0.0) + ln, neg = fmax(-h, 0.0) + ln; // of h and of -h
            const double up = h >= 0.0 ? 1.0 / (1.0 + t) : t / (1.0 + t);    // sigmoid(h)
            const double down = h >= 0.0 ? t / (1.0 + t) : 1.0 / (1.0 + t);
            l = (1.0 - a.smoothing) * neg + a.smoothing * pos;
            dl = a.smoothing * up - (1.0 - a.smoothing) * down;
        } else if (a.kind == RED_PREF_HINGE) {
            l = h >= 1.0 ? 0.0 : 1.0 - h;
            dl = h >= 1.0 ? 0.0 : -1.0;
        } else {
            const double d = (h - 0.5) / a.beta;
            l = d * d;
            dl = 2.0 * d / a.beta;
        }
        const double g = w != 0.0 ? w * dl * a.beta : 0.0;
        loss = w != 0.0 ? w * l : 0.0;
        slope[0] = (float)(g / rows[0]);
        slope[1] = (float)(-g / rows[1]);
    }
    // By one thread: the pair's outputs.
    __device__ __forceinline__ void put(const PairArgs& a, uint32_t p) const
    {
        a.seq_logp[p] = (float)seq[0];
        a.seq_logp[(uint64_t)a.pairs + p] = (float)seq[1];
        a.join.put(p, loss);
    }
};

// Up to kJoinedPairs pairs need no kernel of their own where rows are few: the
// wave of the row that is the last of its pair to have its log-probability
// sums the pair's sequences.  A lane holds one of the 2 P + 1 bounds.
constexpr uint32_t kJoinedPairs = 31;
constexpr uint32_t kPairCounts = kCounterWords - kJoinedPairs * kCountStride;

struct PairJoin {
    const PairArgs& a;
    int bound;             // this lane's, moved into [0, rows] and never falling
    int pair = -1;         // the row's, -1: no sequence has it
    uint32_t expected = 0; // the pair's rows

    // start: this lane's entry of starts (any value past the last)
    __device__ __forceinline__ PairJoin(const PairArgs& args, int64_t start) : a(args)
    {
        const int lane = threadIdx.x & 63;
        bound = start < 0 ? 0 : start > a.rows ? (int)a.rows : (int)start;
        bound = lane <= 2 * (int)a.pairs ? bound : 0x7fffffff;
    }
    __device__ __forceinline__ int rows_of(int p) const
    {
        const int P = (int)a.pairs;
        return __shfl(bound, p + 1) - __shfl(bound, p) + __shfl(bound, P + p + 1) -
               __shfl(bound, P + p);
    }
    __device__ __forceinline__ unsigned arrive(uint32_t row)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int step = 1; step < 64; step *= 2) {
            const int before = __shfl_up(bound, step);
            bound = lane >= step && before > bound ? before : bound;
        }
        const int seq = __popcll(__builtin_amdgcn_ballot_w64(bound <= (int)row)) - 1;
        unsigned before = 0;
        if (seq >= 0 && seq < 2 * (int)a.pairs) {
            pair = seq < (int)a.pairs ? seq : seq - (int)a.pairs;
            expected = (uint32_t)rows_of(pair);
            if (lane == 0)
                before = count_shared(a.counts + pair * kCountStride);
        }
        return before;
    }
    __device__ __forceinline__ void finish(unsigned before, uint32_t row, uint32_t)
    {
        const int lane = threadIdx.x & 63;
        if (pair < 0) {
            if (lane == 0)
                a.row_slope[row] = 0.0f;
        } else if (__builtin_amdgcn_readfirstlane(before) == expected - 1) {
            if (lane == 0)
                clear_shared(a.counts + pair * kCountStride);
            one(pair);
        }
        if (row == 0) // no row of an empty pair will come
            for (int p = 0; p < (int)a.pairs; ++p)
                if (rows_of(p) == 0)
                    one(p);
    }

  private:
    __device__ __forceinline__ void one(int p)
    {
        const int lane = threadIdx.x & 63;
        const PairValues values(a, (uint32_t)p);
        int begin[2], end[2];
        double sum[2], count[2];
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            begin[side] = __shfl(bound, side * (int)a.pairs + p);
            end[side] = __shfl(bound, side * (int)a.pairs + p + 1);
            double s = 0.0, n = 0.0;
            for (int r = begin[side] + lane; r < end[side]; r += 4 * kWave) {
                double x[4];
                int64_t y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool in = r + k * kWave < end[side];
                    x[k] = in ? load_shared(a.row_logp + r + k * kWave) : 0.0;
                    y[k] = in ? a.targets[r + k * kWave] : -1;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s += x[k]; // 0 where the target is not a column
                    n += (uint64_t)y[k] < (uint64_t)a.V ? 1.0 : 0.0;
                }
            }
            sum[side] = s;
            count[side] = n;
        }
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            sum[side] = wave_sum64(sum[side]);
            count[side] = wave_sum64(count[side]);
        }
        const PairResult result(a, values, sum, count);
        if (lane == 0)
            result.put(a, (uint32_t)p);
        const unsigned before = a.join.arrive((uint32_t)p);
#pragma unroll
        for (int side = 0; side < 2; ++side)
            for (int r = begin[side] + lane; r < end[side]; r += kWave)
                a.row_slope[r] = result.slope[side];
        a.join.finish(before, (uint32_t)p, a.pairs);
    }
};

// The pairs by a kernel of their own (rowloss.hip).
hipError_t launch_preference_pairs(const PairArgs& args, hipStream_t stream);

} // namespace red
