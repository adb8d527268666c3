// gdn_rope.cu -- rotary positions of the attention layers' queries and keys (gdn_rope).
//
// Pair i of the first rot elements of a head, at position p:
//   (a, b) -> m (a cos t - b sin t, b cos t + a sin t),   t = p f_i,
// with f_i from gdn_rope_plan_init (theta^(-2i/rot), slowed down for contexts longer than the trained one).
//
// Angles.  f_i is kept as turns per position in units of 2^-64: p f_i modulo whole turns is then the low 64 bits of
// an integer product, exact however far the position (a float's p f_i is off by a radian at p = 10^7).  Its upper 32
// bits are the angle; the nearest quarter turn is taken off them as an integer too, because a float has 24 bits: half a
// turn less 2^-20 would be off by 2^-26 of a turn, 2^-6 of its sine.  What is left, an eighth of a turn at most, is a
// float to 2^-24 of itself.  The frequency has the 53 bits of a double: with the roundings on the way to it below 2^-52 p
// of a turn, over the factor where that is below 1.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_tma.cuh"

namespace gdn {
namespace {

constexpr int kRopeThreads = 256;

// 8 consecutive elements
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void ld(const void* p) { r = *static_cast<const uint4*>(p); }
    __device__ __forceinline__ void st(void* p) const { *static_cast<uint4*>(p) = r; }
    __device__ __forceinline__ void get(float v[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float v[8]) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void ld(const void* p) {
        a = static_cast<const float4*>(p)[0];
        b = static_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void st(void* p) const {
        static_cast<float4*>(p)[0] = a;
        static_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void get(float v[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void set(const float v[8]) {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
};

// sine and cosine of p turns / 2^64 of a turn
__device__ __forceinline__ void sine_cosine(unsigned long long p, unsigned long long turns, float* sn, float* cs) {
    const unsigned a = (unsigned)((p * turns) >> 32), quarter = (a + 0x20000000u) >> 30;
    float s, c;
    sincospif((float)(int)(a - (quarter << 30)) * 0x1p-31f, &s, &c);
    const float s1 = quarter & 1u ? c : s, c1 = quarter & 1u ? s : c;
    *sn = quarter & 2u ? -s1 : s1;
    *cs = (quarter + 1u) & 2u ? -c1 : c1;
}

// A thread owns one piece of 16 elements of a token's heads: 8 pairs of the rotated part (two runs of 8 elements, rot / 2
// apart or side by side), or 16 elements of the rest, which are only copied and only where the result goes elsewhere.  It
// walks over every step_h-th head, kRopeHeads of them in flight; pieces are fastest among the threads, then heads, so that a
// warp's accesses are contiguous.
// MANY tokens: a thread walks over all heads (step_h 1) and makes its 8 angles by itself.  Else the heads are split over
// more threads, and the CTA makes the angles of its tokens once, in shared memory, while the loads are under way: made by
// every thread for its own heads they took 2 us of the 5 that 300 tokens of 26 heads then needed.  (The barrier costs more
// than the angles where there are many tokens: 197 us against 190 for 65536 tokens of 36 heads.)
template <typename T, bool MANY>
__global__ void __launch_bounds__(kRopeThreads, 2) k_rope(const __grid_constant__ RopeJob J) {
    constexpr int kRopeHeads = MANY ? 4 : 2;  // heads whose loads a thread has in flight
    // a CTA's threads reach over at most kRopeThreads / pieces + 2 tokens of rot / 2 <= 8 pieces angles
    __shared__ float2 angle[MANY ? 1 : 8 * kRopeThreads + 2 * 128];  // cosine and sine
    griddep_wait();                                       // launched with programmatic serialization
    griddep_launch_dependents();
    const int pieces = J.pieces, pairs = J.rot / 16, half_rot = J.rot / 2, heads = J.hq + J.hkv;
    // (the launcher keeps these in 32 bits: six divisions of 64 bits took longer than everything else of a small call)
    const unsigned at0 = blockIdx.x * kRopeThreads, at = at0 + threadIdx.x, per_tok = (unsigned)(pieces * J.step_h);
    const unsigned tok0 = at0 / per_tok, tok1 = min((at0 + kRopeThreads - 1) / per_tok, (unsigned)J.n_tok - 1);
    const int64_t tok = at / per_tok;
    const unsigned in_tok = at - (unsigned)tok * per_tok;
    const int h0 = (int)(in_tok / (unsigned)pieces), u = (int)(in_tok - (unsigned)h0 * pieces);
    const bool mine = tok < J.n_tok, turn = u < pairs;
    const int e0 = turn ? (J.half ? 8 * u : 16 * u) : J.rot + 16 * (u - pairs);
    const int e1 = e0 + (turn && J.half ? half_rot : 8);
    const bool two = e1 < J.D;  // (a head's rest may end on a single run)
    auto in_place = [&](int h) { return h < J.hq ? J.q == J.q_out : J.k == J.k_out; };
    float c[8], s[8];
    for (int hb = h0;; hb += kRopeHeads * J.step_h) {
        Eight<T> x[kRopeHeads], y[kRopeHeads];
#pragma unroll
        for (int e = 0; e < kRopeHeads; ++e) {
            const int h = hb + e * J.step_h;
            if (!mine || h >= heads || (!turn && in_place(h))) continue;
            const T* src = h < J.hq ? static_cast<const T*>(J.q) + tok * J.ldq + (int64_t)h * J.D
                                    : static_cast<const T*>(J.k) + tok * J.ldk + (int64_t)(h - J.hq) * J.D;
            x[e].ld(src + e0);
            if (two) y[e].ld(src + e1);
        }
        if (hb == h0 && MANY) {
            if (!mine) return;
            const unsigned long long p = (unsigned long long)(long long)J.positions[tok];
            if (turn)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sine_cosine(p, J.turns[8 * u + j], &s[j], &c[j]);
                    c[j] *= J.mscale;
                    s[j] *= J.mscale;
                }
        }
        if (hb == h0 && !MANY) {
            for (unsigned j = threadIdx.x; j < (tok1 - tok0 + 1) * half_rot; j += kRopeThreads) {
                const unsigned t = j / (unsigned)half_rot;
                const unsigned long long p = (unsigned long long)(long long)J.positions[tok0 + t];
                float sn, cs;
                sine_cosine(p, J.turns[j - t * half_rot], &sn, &cs);
                angle[j] = make_float2(cs * J.mscale, sn * J.mscale);
            }
            __syncthreads();
            if (!mine) return;
            if (turn)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 w = angle[(int)(tok - tok0) * half_rot + 8 * u + j];
                    c[j] = w.x;
                    s[j] = w.y;
                }
        }
#pragma unroll
        for (int e = 0; e < kRopeHeads; ++e) {
            const int h = hb + e * J.step_h;
            if (h >= heads || (!turn && in_place(h))) continue;
            T* dst = h < J.hq ? static_cast<T*>(J.q_out) + tok * J.ldqo + (int64_t)h * J.D
                              : static_cast<T*>(J.k_out) + tok * J.ldko + (int64_t)(h - J.hq) * J.D;
            if (turn) {
                float a[8], b[8];
                x[e].get(a);
                y[e].get(b);
                if (J.half) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float a1 = a[j] * c[j] - b[j] * s[j];
                        b[j] = b[j] * c[j] + a[j] * s[j];
                        a[j] = a1;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a1 = a[2 * j] * c[j] - a[2 * j + 1] * s[j];
                        a[2 * j + 1] = a[2 * j + 1] * c[j] + a[2 * j] * s[j];
                        a[2 * j] = a1;
                        const float b1 = b[2 * j] * c[j + 4] - b[2 * j + 1] * s[j + 4];
                        b[2 * j + 1] = b[2 * j + 1] * c[j + 4] + b[2 * j] * s[j + 4];
                        b[2 * j] = b1;
                    }
                }
                x[e].set(a);
                y[e].set(b);
            }
            x[e].st(dst + e0);
            if (two) y[e].st(dst + e1);
        }
        if (hb + kRopeHeads * J.step_h >= heads) return;
    }
}

}  // namespace

// theta^(-2i/rot) / 2 pi in turns, slowed down by `factor` (orig_len 0: every pair; else by parts: pairs that turn more than
// beta_fast times within orig_len positions keep their frequency, those that turn less than beta_slow times are slowed down, a
// ramp over the pairs joins them), as multiples of 2^-64
void rope_turns(int rot, double theta, double factor, int orig_len, double beta_fast, double beta_slow, uint64_t* turns) {
    constexpr double two_pi = 6.283185307179586476925286766559;
    double low = 0.0, high = 0.0;
    if (orig_len > 0) {
        auto pair_of = [&](double n) { return rot * std::log(orig_len / (n * two_pi)) / (2.0 * std::log(theta)); };
        low = std::max(std::floor(pair_of(beta_fast)), 0.0);
        high = std::min(std::ceil(pair_of(beta_slow)), rot - 1.0);
    }
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rot);
        if (orig_len > 0) {
            const double ramp = std::min(std::max((i - low) / std::max(high - low, 0.001), 0.0), 1.0);
            f = f * (1.0 - ramp) + f / factor * ramp;
        } else {
            f /= factor;
        }
        // whole turns per position (of a factor far below 1) are none
        const double t = f / two_pi;
        turns[i] = (uint64_t)std::llround((t - std::floor(t)) * 0x1p62) << 2;
    }
}

cudaError_t launch_rope(RopeJob job, cudaStream_t st) {
    const int heads = job.hq + job.hkv, es = job.bf16 ? 2 : 4;
    const bool same = job.q == job.q_out && job.k == job.k_out;
    job.pieces = job.rot / 16 + (same ? 0 : (job.D - job.rot + 15) / 16);
    auto at = [&](const void* p, int64_t ld, int64_t tok) {
        return p ? static_cast<const unsigned char*>(p) + tok * ld * es : nullptr;
    };
    auto out_at = [&](void* p, int64_t ld, int64_t tok) { return p ? static_cast<unsigned char*>(p) + tok * ld * es : nullptr; };
    // one thread per piece and token walks all heads once that fills the GPU (512 threads an SM); fewer tokens split the
    // heads.  Thread numbers stay in 32 bits: 2^22 tokens of 16 pieces a launch.
    constexpr int64_t kTokens = (int64_t)1 << 22;
    for (int64_t first = 0; first < job.n_tok && heads > 0; first += kTokens) {
        RopeJob J = job;
        J.n_tok = std::min(kTokens, job.n_tok - first);
        J.positions += first;
        J.q = at(job.q, job.ldq, first);
        J.k = at(job.k, job.ldk, first);
        J.q_out = out_at(job.q_out, job.ldqo, first);
        J.k_out = out_at(job.k_out, job.ldko, first);
        const int64_t full = (int64_t)sm_count() * 512, one = J.n_tok * J.pieces;
        J.step_h = (int)std::min<int64_t>(heads, std::max<int64_t>(1, full / one));
        const dim3 grid((unsigned)((one * J.step_h + kRopeThreads - 1) / kRopeThreads));
        const auto kernel = J.step_h == 1 ? (J.bf16 ? k_rope<__nv_bfloat16, true> : k_rope<float, true>)
                                          : (J.bf16 ? k_rope<__nv_bfloat16, false> : k_rope<float, false>);
        const cudaError_t e = launch_pdl(kernel, grid, dim3(kRopeThreads), 0, st, J);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace gdn
