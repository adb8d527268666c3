// gdn_rope.cu -- rotary positions of the attention layers' queries and keys (gdn_rope).
//
// Pair i of the first rot elements of a head, at position p:
//   (a, b) -> m (a cos t - b sin t, b cos t + a sin t),   t = p f_i,
// with f_i from gdn_rope_plan_init (theta^(-2i/rot), slowed down for contexts longer than the trained one).
//
// Angles.  f_i is kept as turns per position in units of 2^-64: p f_i modulo whole turns is then the low 64 bits of
// an integer product, exact however far the position (a float's p f_i is off by a radian at p = 10^7), and its
// upper 32 bits as a signed number are the angle in (-1/2, 1/2] turns for sincospif.  The frequency itself has the 53
// bits of a double: 2^-54 p of a turn, 2^-34 at a position of 2^20.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_tma.cuh"

namespace gdn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;  // pieces whose loads a thread has in flight

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

// A CTA takes a few tokens: its threads make their sines and cosines once, into shared memory, and then rotate the heads
// from there.  (With every thread making its own angles for one head, sine and cosine took longer than the memory; with a
// thread walking over the heads of one angle, few tokens leave the GPU empty.)  The unit of work is a piece of 16 elements of a head: 8 pairs
// of the rotated part (two runs of 8 elements, rot / 2 apart or side by side), or 16 elements of the rest, which are only
// copied and only where the result goes elsewhere.  Pieces are fastest among the threads, then heads, so that a warp's
// accesses are contiguous; the first loads are under way while the angles are made.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const __grid_constant__ RopeJob J) {
    extern __shared__ float2 angle[];  // [token][rot / 2]: cosine and sine
    griddep_wait();                    // launched with programmatic serialization
    griddep_launch_dependents();
    const int pieces = J.pieces, pairs = J.rot / 16, heads = J.hq + J.hkv, half_rot = J.rot / 2;
    const int64_t first = (int64_t)blockIdx.x * J.per_cta;
    const int n = (int)(J.n_tok - first < J.per_cta ? J.n_tok - first : J.per_cta);
    const int items = n * heads * pieces, step = (int)gridDim.y * kRopeThreads;
    bool ready = false;
    for (int i0 = (int)blockIdx.y * kRopeThreads + (int)threadIdx.x; !ready || i0 < items; i0 += kRopeUnroll * step) {
        Eight<T> x[kRopeUnroll], y[kRopeUnroll];
        T* dst[kRopeUnroll];
        int at[kRopeUnroll], e1[kRopeUnroll];  // the angles (-1: none), the second run's distance (0: none)
#pragma unroll
        for (int e = 0; e < kRopeUnroll; ++e) {
            const int i = i0 + e * step;
            dst[e] = nullptr;
            if (i >= items) continue;
            const int row = i / pieces, u = i - row * pieces, t = row / heads, h = row - t * heads;
            const int64_t tok = first + t;
            int e0;
            if (u < pairs) {
                e0 = J.half ? 8 * u : 16 * u;
                e1[e] = J.half ? half_rot : 8;
                at[e] = t * half_rot + 8 * u;
            } else {
                e0 = J.rot + 16 * (u - pairs);
                e1[e] = e0 + 8 < J.D ? 8 : 0;  // (a head's rest may end on a single run)
                at[e] = -1;
            }
            const bool q = h < J.hq;
            const int64_t off = (int64_t)(q ? h : h - J.hq) * J.D + e0;
            const T* src = static_cast<const T*>(q ? J.q : J.k) + tok * (q ? J.ldq : J.ldk) + off;
            dst[e] = static_cast<T*>(q ? J.q_out : J.k_out) + tok * (q ? J.ldqo : J.ldko) + off;
            x[e].ld(src);
            if (e1[e]) y[e].ld(src + e1[e]);
        }
        if (!ready) {
            for (int j = threadIdx.x; j < n * half_rot; j += kRopeThreads) {
                const int t = j / half_rot;
                const unsigned long long p = (unsigned long long)(long long)J.positions[first + t];
                const int turn = (int)(unsigned)((p * J.turns[j - t * half_rot]) >> 32);
                float s, c;
                sincospif((float)turn * 0x1p-31f, &s, &c);
                angle[j] = make_float2(c * J.mscale, s * J.mscale);
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int e = 0; e < kRopeUnroll; ++e) {
            if (!dst[e]) continue;
            if (at[e] >= 0) {
                float a[8], b[8], c[8], s[8];
                x[e].get(a);
                y[e].get(b);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 w = *reinterpret_cast<const float4*>(angle + at[e] + 2 * j);
                    c[2 * j] = w.x, s[2 * j] = w.y, c[2 * j + 1] = w.z, s[2 * j + 1] = w.w;
                }
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
            x[e].st(dst[e]);
            if (e1[e]) y[e].st(dst[e] + e1[e]);
        }
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
        turns[i] = (uint64_t)std::llround(f / two_pi * 0x1p62) << 2;  // (f <= 1: below a sixth of a turn)
    }
}

cudaError_t launch_rope(RopeJob job, cudaStream_t st) {
    const int heads = job.hq + job.hkv;
    if (job.n_tok == 0 || heads == 0) return cudaSuccess;
    const bool same = job.q == job.q_out && job.k == job.k_out;
    job.pieces = job.rot / 16 + (same ? 0 : (job.D - job.rot + 15) / 16);
    // Tokens of a CTA: angles for its threads to make and a few pieces for each of them; one token where the tokens would not
    // fill the GPU's CTAs (8 an SM) otherwise.  A token of very many pieces is shared by CTAs along y.
    const int per_token = heads * job.pieces;
    job.per_cta = std::max(1, std::min(2 * kRopeThreads / job.rot, 4 * kRopeThreads / per_token));
    if (job.n_tok < (int64_t)sm_count() * 8 * job.per_cta) job.per_cta = 1;
    const dim3 grid((unsigned)((job.n_tok + job.per_cta - 1) / job.per_cta),
                    (unsigned)((job.per_cta * per_token + 8 * kRopeThreads - 1) / (8 * kRopeThreads)));
    const size_t smem = (size_t)job.per_cta * (job.rot / 2) * sizeof(float2);
    return job.bf16 ? launch_pdl(k_rope<__nv_bfloat16>, grid, dim3(kRopeThreads), smem, st, job)
                    : launch_pdl(k_rope<float>, grid, dim3(kRopeThreads), smem, st, job);
}

}  // namespace gdn
