// threshold.cuh -- the threshold of a 1.5-entmax row from repeated sums over its scores, shared by the serving
// kernels (prompt.cu, cache_attn.cu).
#pragma once

namespace entmax {

// The threshold iteration of 1.5-entmax for one row: the root t of g(t) = sum max(0, S - t)^2 = 4, from sums
// over the scores above the present t.
//   Newton's step is a lower bound of the root from either side (g is convex and decreasing); its error is of
//   second order, (e / d)^2 / 2 for an error e before and a mean depth d = s2 / s1 of the support.
//   The root of sum_{S > t} (S - r)^2 = 4, t + mean - sqrt(4 / k - variance), is exact once {S > t} is the
//   support; otherwise its error is that of the few scores between t and the root: (e / d)^3 / 6 where they
//   lie dense, (e / d)^2 / 2 where one does.
// So the closed form where it lies above the bound, and the bound where not, or from pass CLOSED on.  Settled
// when the step shows that what is left is about 1e-5 d at most, and 1e-7 d as a rule.
constexpr float STEP_CLOSED = 5e-3f, STEP_NEWTON = 1e-3f;
constexpr int CLOSED = 8, MOST_PASSES = 40;
struct Threshold {
    float t, lo;
    bool settled;
    __device__ __forceinline__ void start(float t0) {
        t = lo = t0;
        settled = false;
    }
    __device__ __forceinline__ void step(float k, float s1, float s2, int pass) {
        if (!(k > 0.f)) {  // above all scores: back to the bound
            settled = !(t > lo);
            t = lo;
            return;
        }
        lo = fmaxf(lo, t + (s2 - 4.f) / (2.f * s1));
        const float mean = s1 / k, rest = 4.f / k - (s2 / k - mean * mean);
        const float root = t + mean - sqrtf(fmaxf(rest, 0.f));
        const bool closed = rest >= 0.f && root >= lo && pass <= CLOSED;
        const float next = closed ? root : lo;
        settled = !(fabsf(next - t) > (closed ? STEP_CLOSED : STEP_NEWTON) * (s2 / s1));
        t = next;
    }
};

}  // namespace entmax
