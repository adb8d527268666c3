// gdn_attn_tree.cu -- attention of a tree of drafted tokens per sequence over its paged KV cache:
// node i attends to the cached tokens 0 .. ctx - 1, to its ancestors and to itself.
#include <cuda_bf16.h>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_tma.cuh"

namespace gdn {
namespace {

// The simple form: a warp per (node, query head), lane = D / 32 consecutive dims, one key at
// a time with a running maximum and sum.
template <int D>
__global__ void __launch_bounds__(128) k_attn_tree(const __grid_constant__ AttnTreeJob J) {
    constexpr int DPL = D / 32;
    griddep_wait();  // launched with programmatic serialization
    griddep_launch_dependents();
    const int i = blockIdx.x, h = blockIdx.y * 4 + (threadIdx.x >> 5), b = blockIdx.z, lane = threadIdx.x & 31;
    const int64_t first = J.cu_nodes[b];
    const int64_t n = (int64_t)J.cu_nodes[b + 1] - first;
    const int ctx = J.ctx_lens[b];
    if (first < 0 || n < 1 || n > J.max_nodes || first + n > J.n_nodes || ctx < 0 || ctx > J.max_ctx ||
        ctx > (int64_t)J.max_pages * J.page || i >= n || h >= J.Hq)
        return;
    const int G = J.Hq / J.Hkv, kvh = h / G;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(J.q) + ((first + i) * J.Hq + h) * D + lane * DPL;
    float qv[DPL], o[DPL], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < DPL; ++e) {
        qv[e] = __bfloat162float(q[e]) * J.scale;
        o[e] = 0.f;
    }
    auto take = [&](const __nv_bfloat16* k, const __nv_bfloat16* v) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < DPL; ++e) s = fmaf(qv[e], __bfloat162float(k[lane * DPL + e]), s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float mn = fmaxf(m, s);
        const float f = m == -INFINITY ? 0.f : __expf(m - mn);
        const float p = __expf(s - (mn == -INFINITY ? 0.f : mn));
        l = l * f + p;
        m = mn;
#pragma unroll
        for (int e = 0; e < DPL; ++e) o[e] = fmaf(p, __bfloat162float(v[lane * DPL + e]), o[e] * f);
    };
    const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(J.k_pool);
    const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(J.v_pool);
    for (int t = 0; t < ctx; ++t) {
        const int id = J.block_table[(size_t)b * J.max_pages + t / J.page];
        if (id < 0 || id >= J.n_pages) continue;
        const size_t at = (((size_t)id * J.Hkv + kvh) * J.page + t % J.page) * D;
        take(kp + at, vp + at);
    }
    for (int a = i; a >= 0;) {
        const size_t at = ((size_t)(first + a) * J.Hkv + kvh) * D;
        take(static_cast<const __nv_bfloat16*>(J.k_new) + at, static_cast<const __nv_bfloat16*>(J.v_new) + at);
        const int p = J.parents[first + a];
        a = p >= 0 && p < a ? p : -1;
    }
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(J.o) + ((size_t)(first + i) * J.Hq + h) * D + lane * DPL;
#pragma unroll
    for (int e = 0; e < DPL; ++e) dst[e] = __float2bfloat16_rn(o[e] / l);
}

}  // namespace

size_t attn_tree_workspace_bytes(int B, int Hq, int Hkv, int D, int max_nodes, int max_ctx) { return 0; }

cudaError_t launch_attn_tree(const AttnTreeJob& j, cudaStream_t st) {
    if (j.B == 0 || j.n_nodes == 0) return cudaSuccess;
    const dim3 grid((unsigned)j.max_nodes, (unsigned)((j.Hq + 3) / 4), (unsigned)j.B);
    if (j.D == 256) return launch_pdl(k_attn_tree<256>, grid, dim3(128), 0, st, j);
    return launch_pdl(k_attn_tree<128>, grid, dim3(128), 0, st, j);
}

}  // namespace gdn
