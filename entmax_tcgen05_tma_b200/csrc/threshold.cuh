// threshold.cuh -- the threshold of a 1.5-entmax row from repeated sums over its scores, shared by the serving
// kernels (prompt.cu, cache_attn.cu).
#pragma once

namespace entmax {

// The threshold iteration of 1.5-entmax for one row: the root t of g(t) = sum max(0, S - t)^2 = 4, from sums
// over the scores above the present t.
//   Newton's step is a lower bound of the root from either side (g is convex and decreasing); its error is of
//   second order, (e / d)^2 / 2 for an error e before and a mean depth d = s2 / s1 of the support.
//   The root of sum_{S > t} (S - r)^2 = 4, t + mean - sqrt(4 / k - variance) with k scores above t, is exact once
//   {S > t} is the support; otherwise its error is that of the few scores between t and the root: (e / d)^3 / 6
//   where they lie dense, at most (e / d)^2 / 2 / k where one does.
// So the closed form where it lies above the bound, and the bound where not, or from pass CLOSED on.  The row is
// settled when the step, in units of d, was at most `step`: 0.02 leaves 2e-6 d as a rule and 5e-5 d at most, 0.005
// 1e-7 and 1e-6, 0.003 a third of that (rows of 33 to 8192 normal scores; with 0.005 the fp32 output of prompts of 33 to
// 256 tokens was off by 9.4e-7, with 0.003 by 3.7e-7).
// Counting k costs as much as both sums, so a caller may leave it out from the second pass on: the sums s1 of two
// passes give the mean count between their t (s1' = -k), and its change from the last gives the count here.
constexpr float STEP_NEWTON = 1e-3f;
constexpr int CLOSED = 8, MOST_PASSES = 40;
struct Threshold {
    float t, lo;
    float t_before, s1_before, k_before;
    bool settled;
    __device__ __forceinline__ void start(float t0) {
        t = lo = t0;
        t_before = s1_before = k_before = 0.f;
        settled = false;
    }
    // k < 0: not counted
    __device__ __forceinline__ void step(float k, float s1, float s2, int pass, float step) {
        if (!(s1 > 0.f)) {  // above all scores: back to the bound
            settled = !(t > lo);
            t = lo;
            return;
        }
        if (k < 0.f) {
            const float mean_k = t != t_before ? __fdividef(s1_before - s1, t - t_before) : k_before;
            k = fmaxf(2.f * mean_k - k_before, __fdividef(s1 * s1, s2));  // at least that, by Cauchy and Schwarz
        }
        t_before = t;
        s1_before = s1;
        k_before = k;
        // quotients and the root to about 2^-22: a few instructions each, in code that mostly runs once a row
        const float per_s1 = __fdividef(1.f, s1), per_k = __fdividef(1.f, k);
        lo = fmaxf(lo, t + 0.5f * (s2 - 4.f) * per_s1);
        const float mean = s1 * per_k, rest = (4.f - s2) * per_k + mean * mean;
        float root;
        asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(fmaxf(rest, 0.f)));
        root = t + __fdividef((s2 - 4.f) * per_k, mean + root);  // = mean - root, which loses digits
        const bool closed = rest >= 0.f && root >= lo && pass <= CLOSED;
        const float next = closed ? root : lo;
        settled = !(fabsf(next - t) > (closed ? step : STEP_NEWTON) * s2 * per_s1);
        t = next;
    }
};

}  // namespace entmax
