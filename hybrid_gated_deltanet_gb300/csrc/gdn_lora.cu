// gdn_lora.cu -- the low side of the adapters beside a shared projection (gdn_proj_lora): v_t = scale_a A_a x_t for every
// token t of a request with adapter a.  The requests are rows cu_rows[s] .. cu_rows[s+1] of the tokens.
#include <cuda_bf16.h>

#include <algorithm>

#include "gdn_internal.h"
#include "gdn_tma.cuh"

namespace gdn {
namespace {

constexpr int kLowThreads = 256;
constexpr int kLowWarps = kLowThreads / 32;
constexpr int kShortRequest = 16;  // tokens from which on the tensor cores take a request of a wide call

// The request that token t belongs to, or -1: the last s with cu[s] <= t, if t < cu[s+1].  By a whole warp, 32 probes a
// round; where every request is one token (decoding) the first guess is right.  Any contents of cu stay in bounds.
__device__ __forceinline__ int request_of(const int32_t* cu, int n, int t, int lane) {
    int lo = -1, hi = n;
    if (t < n && cu[t] <= t && t < cu[t + 1]) {
        lo = t;
        hi = t + 1;
    }
    while (hi - lo > 1) {
        const int step = (hi - lo + 32) / 33;
        const int64_t p = (int64_t)lo + (int64_t)(lane + 1) * step;
        const unsigned m = __ballot_sync(0xffffffffu, p < hi && cu[p < hi ? p : 0] <= t);
        lo += __popc(m) * step;
        hi = min(hi, lo + step);
    }
    return lo >= 0 && cu[lo] >= 0 && cu[lo] <= t && t < cu[lo + 1] ? lo : -1;
}

// v by dot products, for tokens that share their adapter with few others or none, so that there is nothing for a matrix
// product to share.  Bound by the adapters' bytes, or by the latency of a pass over a row when there are few: a warp
// makes ROWS rows of A for a token, all its loads independent.
template <int ROWS, typename Store>
__device__ __forceinline__ void low_rows(const LowJob& J, int64_t t, int a, int j0, int cols, Store store) {
    const int K = J.k, rank = J.rank, lane = threadIdx.x & 31;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(J.x) + t * K;
    const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(J.a) + ((int64_t)a * rank + j0) * K;
    const float scale = J.scale ? J.scale[a] : 1.f;
    float acc[ROWS] = {};
#pragma unroll 8
    for (int c = 8 * lane; c < K; c += 256) {
        const uint4 xv = *reinterpret_cast<const uint4*>(x + c);
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (j0 + r >= rank) break;
            const uint4 av = *reinterpret_cast<const uint4*>(A + (int64_t)r * K + c);
            const uint32_t aw[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[r] = fmaf(__uint_as_float(xw[e] << 16), __uint_as_float(aw[e] << 16), acc[r]);
                acc[r] = fmaf(__uint_as_float(xw[e] & 0xffff0000u), __uint_as_float(aw[e] & 0xffff0000u), acc[r]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
        if (lane == 0 && j0 + r < cols) store(j0 + r, j0 + r < rank ? acc[r] * scale : 0.f);
    }
}

// few tokens: a CTA per token and 8 rows of A, fp32 results
__global__ void __launch_bounds__(kLowThreads) k_lora_low(const __grid_constant__ LowJob J) {
    griddep_wait();  // launched with programmatic serialization
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = (int)blockIdx.x;
    const int s = request_of(J.cu_rows, J.n_seg, t, lane);
    int a = s >= 0 ? J.adapter_idx[s] : -1;
    if (a < 0 || a >= J.n_adapters) a = -1;
    if (threadIdx.x == 0 && blockIdx.y == 0) J.tok_adapter[t] = a;
    const int j = (int)blockIdx.y * kLowWarps + warp;
    if (a < 0 || j >= J.rank) return;
    float* v = static_cast<float*>(J.v) + (int64_t)t * J.rank;
    low_rows<1>(J, t, a, j, J.rank, [&](int c, float x) { v[c] = x; });
}

// many tokens: a CTA per request and 16 rows of A.  Requests below kShortRequest tokens get their v here (as hi + lo), the
// longer ones from the tensor cores behind this kernel; the first and the last request's CTAs also mark what lies outside.
__global__ void __launch_bounds__(kLowThreads) k_lora_short(const __grid_constant__ LowJob J) {
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, s = (int)blockIdx.x, n_tok = (int)J.n_tok;
    int first = 0, last = 0, a = -1;
    if (J.n_seg > 0) {
        first = min(max(J.cu_rows[s], 0), n_tok);
        last = min(max(J.cu_rows[s + 1], 0), n_tok);
        a = J.adapter_idx[s];
    }
    if (a < 0 || a >= J.n_adapters) a = -1;
    const bool later = last - first >= kShortRequest;
    if (blockIdx.y == 0) {
        const int mark = a >= 0 && later ? a | kLongRequest : a;
        for (int t = first + threadIdx.x; t < last; t += kLowThreads) J.tok_adapter[t] = mark;
        if (s == 0)
            for (int t = threadIdx.x; t < first; t += kLowThreads) J.tok_adapter[t] = -1;
        if (s >= J.n_seg - 1)
            for (int t = last + threadIdx.x; t < n_tok; t += kLowThreads) J.tok_adapter[t] = -1;
    }
    if (a < 0 || later) return;
    const int cols = (J.rank + 15) / 16 * 16, row = low_row(J.rank), lo = J.rank <= 32 ? cols : row / 2;
    const int j0 = ((int)blockIdx.y * kLowWarps + warp) * 2;
    if (j0 >= cols) return;
    for (int t = first; t < last; ++t) {
        __nv_bfloat16* v = static_cast<__nv_bfloat16*>(J.v) + (int64_t)t * row;
        low_rows<2>(J, t, a, j0, cols, [&](int c, float x) {
            const __nv_bfloat16 hi = __float2bfloat16_rn(x);
            const float h = __bfloat162float(hi);
            v[c] = hi;
            v[lo + c] = __float2bfloat16_rn(isfinite(h) ? x - h : 0.f);
        });
    }
}

}  // namespace

cudaError_t launch_lora_low(const LowJob& job, cudaStream_t st) {
    if (job.n_tok == 0) return cudaSuccess;
    if (job.wide) {
        const dim3 grid((unsigned)std::max(job.n_seg, 1), (unsigned)((job.rank + 2 * kLowWarps - 1) / (2 * kLowWarps)));
        return launch_pdl(k_lora_short, grid, dim3(kLowThreads), 0, st, job);
    }
    const dim3 grid((unsigned)job.n_tok, (unsigned)((job.rank + kLowWarps - 1) / kLowWarps));
    return launch_pdl(k_lora_low, grid, dim3(kLowThreads), 0, st, job);
}

}  // namespace gdn
