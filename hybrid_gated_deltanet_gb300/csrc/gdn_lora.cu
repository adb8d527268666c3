// gdn_lora.cu -- the low side of the adapters beside a shared projection (gdn_proj_lora): v_t = scale_a A_a x_t for every
// token t of a request with adapter a.  The requests are rows cu_rows[s] .. cu_rows[s+1] of the tokens.
#include <cuda_bf16.h>

#include <algorithm>

#include "gdn_common.cuh"
#include "gdn_gemm.cuh"
#include "gdn_internal.h"
#include "gdn_tc.cuh"
#include "gdn_tma.cuh"

namespace gdn {
namespace {

constexpr int kLowThreads = 256;
constexpr int kLowWarps = kLowThreads / 32;
constexpr int kShortRequest = 16;  // tokens from which on the tensor cores take a request of a wide call

// The request that token t belongs to, or -1: the last s with cu[s] <= t, if t < cu[s+1].  By a whole warp, 32 probes a
// round; where every request is one token (decoding) the first guess is right.  Any contents of cu stay in bounds.
__device__ __forceinline__ int request_of(const int32_t* cu, int n, int t, int lane, int64_t& len) {
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
    len = 0;
    if (lo < 0) return -1;
    const int first = cu[lo], last = cu[lo + 1];
    if (first < 0 || t < first || t >= last) return -1;
    len = (int64_t)last - first;
    return lo;
}

// v by dot products, a warp for ROWS rows of A at a time: tokens of requests short enough that every token (nearly) reads
// an adapter of its own, so that there is nothing for a matrix product to share.  Bound by the adapters' bytes, or by the
// latency of one pass over a row when there are few.
template <int ROWS, bool WIDE>
__global__ void __launch_bounds__(kLowThreads) k_lora_low(const __grid_constant__ LowJob J) {
    __shared__ int s_adapter[kLowWarps];
    griddep_wait();  // launched with programmatic serialization
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = (int64_t)blockIdx.x * J.per_cta;
    if (warp < J.per_cta) {
        const int64_t t = first + warp;
        int a = -1;
        if (t < J.n_tok) {
            int64_t len;
            const int s = request_of(J.cu_rows, J.n_seg, (int)t, lane, len);
            if (s >= 0) a = J.adapter_idx[s];
            if (a < 0 || a >= J.n_adapters) a = -1;
            const bool later = J.wide && a >= 0 && len >= kShortRequest;
            if (lane == 0 && blockIdx.y == 0) J.tok_adapter[t] = later ? a | kLongRequest : a;
            if (later) a = -1;
        }
        if (lane == 0) s_adapter[warp] = a;
    }
    __syncthreads();
    const int K = J.k, rank = J.rank, cols = WIDE ? (rank + 15) / 16 * 16 : rank;
    for (int i = 0; i < J.per_cta; ++i) {
        const int a = s_adapter[i];
        if (a < 0) continue;
        const int64_t t = first + i;
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(J.x) + t * K;
        const float scale = J.scale ? J.scale[a] : 1.f;
        for (int j0 = ((int)blockIdx.y * kLowWarps + warp) * ROWS; j0 < cols; j0 += (int)gridDim.y * kLowWarps * ROWS) {
            const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(J.a) + ((int64_t)a * rank + j0) * K;
            float acc[ROWS] = {};
#pragma unroll 4
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
                if (lane != 0 || j0 + r >= cols) continue;
                const float v = j0 + r < rank ? acc[r] * scale : 0.f;
                if (WIDE) {  // v = hi + lo
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(J.v) + t * low_row(rank) + j0 + r;
                    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                    const float h = __bfloat162float(hi);
                    dst[0] = hi;
                    dst[rank <= 32 ? cols : low_row(rank) / 2] = __float2bfloat16_rn(isfinite(h) ? v - h : 0.f);
                } else {
                    static_cast<float*>(J.v)[t * rank + j0 + r] = v;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_lora_low(LowJob job, cudaStream_t st) {
    if (job.n_tok == 0) return cudaSuccess;
    if (job.wide) {
        job.per_cta = kLowWarps;
        const dim3 grid((unsigned)((job.n_tok + kLowWarps - 1) / kLowWarps));
        return launch_pdl(k_lora_low<2, true>, grid, dim3(kLowThreads), 0, st, job);
    }
    job.per_cta = 1;
    const dim3 grid((unsigned)job.n_tok, (unsigned)((job.rank + kLowWarps - 1) / kLowWarps));
    return launch_pdl(k_lora_low<1, false>, grid, dim3(kLowThreads), 0, st, job);
}

}  // namespace gdn
