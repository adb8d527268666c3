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
    return lo >= 0 && cu[lo] <= t && t < cu[lo + 1] ? lo : -1;
}

// v by dot products, for tokens that share their adapter with few others or none, so that there is nothing for a matrix
// product to share.  Bound by the adapters' bytes, or by the latency of a pass over a row when there are few: a warp
// makes ROWS rows of A for a token, all its loads independent.
// 16 bytes, or zeros; volatile, so that all loads of a round are on their way before the first is used
__device__ __forceinline__ uint4 ld16_if(bool there, const void* p) {
    uint4 v;
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
        " @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((int)there)
        : "memory");
    return v;
}

template <int ROWS, typename Store>
__device__ __forceinline__ void low_rows(const LowJob& J, int64_t t, int a, int j0, int cols, Store store) {
    constexpr int U = ROWS == 1 ? 16 : 8;  // pieces of 256 elements in flight
    const int K = J.k, rank = J.rank, lane = threadIdx.x & 31;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(J.x) + t * K;
    const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(J.a) + ((int64_t)a * rank + j0) * K;
    const float scale = J.scale ? J.scale[a] : 1.f;
    float acc[ROWS] = {};
    for (int c0 = 8 * lane; c0 < K; c0 += 256 * U) {
        uint4 xv[U], av[U][ROWS];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = c0 + 256 * i;
            xv[i] = ld16_if(c < K, x + c);
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                av[i][r] = ld16_if(c < K && j0 + r < rank, A + (int64_t)r * K + c);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const uint32_t xw[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const uint32_t aw[4] = {av[i][r].x, av[i][r].y, av[i][r].z, av[i][r].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[r] = fmaf(__uint_as_float(xw[e] << 16), __uint_as_float(aw[e] << 16), acc[r]);
                    acc[r] = fmaf(__uint_as_float(xw[e] & 0xffff0000u), __uint_as_float(aw[e] & 0xffff0000u), acc[r]);
                }
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
__global__ void __launch_bounds__(kLowThreads, 2) k_lora_low(const __grid_constant__ LowJob J) {
    griddep_wait();  // launched with programmatic serialization
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = (int)blockIdx.x;
    const int likely = t < J.n_seg ? J.adapter_idx[t] : -1;  // (asked for beside cu_rows, not behind it)
    const int s = request_of(J.cu_rows, J.n_seg, t, lane);
    int a = s == t ? likely : s >= 0 ? J.adapter_idx[s] : -1;
    if (a < 0 || a >= J.n_adapters) a = -1;
    if (threadIdx.x == 0 && blockIdx.y == 0) J.tok_adapter[t] = a;
    const int j = (int)blockIdx.y * kLowWarps + warp;
    if (a < 0 || j >= J.rank) return;
    float* v = static_cast<float*>(J.v) + (int64_t)t * J.rank;
    low_rows<1>(J, t, a, j, J.rank, [&](int c, float x) { v[c] = x; });
}

// ---- many tokens -----------------------------------------------------------------------------------
// One launch of two kinds of CTAs.  Requests of kShortRequest tokens and more: a cluster per 128 tokens, the tokens being
// the MMA's M side (TMEM lanes) and the rank its N side; the MMAs of an adapter leave the lanes of other tokens as they are
// (lane mask).  The product is small and its tokens are read once per adapter of a tile, so it is bound by its latency: K
// is split over the cluster until the GPU is full, and the fp32 parts are joined through distributed shared memory in
// the order of the ranks, each CTA finishing its share of the tokens.  Shorter requests: a CTA per request and 12 rows
// of A, dot products as above; these CTAs also write down each token's adapter for the projection that follows.
constexpr int kLowTcThreads = 192;
constexpr int kLowTcWarps = kLowTcThreads / 32;
constexpr int kLowK = 64;
constexpr int kXBytes = 128 * kLowK * 2;
constexpr int kLowRing = 6 * kXBytes;      // stages of x and, at most as many, rows of A; then the partial block
constexpr int kLowCu = 1024;               // requests whose ends are searched in shared memory
constexpr int kLowCuOff = kLowRing;
constexpr int kLowBar = kLowCuOff + (kLowCu + 1) * 4 + 4;  // full[5], empty[5], done, TMEM address
constexpr int kLowSmem = kLowBar + 11 * 8 + 8 + 1024;
static_assert(2 * (kLowSmem + 1024) <= 227 * 1024 && 128 * 128 * 4 <= kLowRing, "two CTAs on an SM, the partial block");

struct WideLowArgs {
    LowJob J;
    int32_t kb, ks, n_split, y_split;  // CTAs [0, n_split): long requests; y_split CTAs per short one
};

__device__ __forceinline__ void mma_bf16_lanes(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc,
                                               const uint32_t off[4]) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %6, %7, %8}, p;\n}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(acc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
        : "memory");
}

__device__ __forceinline__ void tma_tile_3d(void* dst, const void* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// v = hi + lo in bf16.  What rounds to infinity is cut to the largest bf16 number first, so that lo can make up for it.
__device__ __forceinline__ void split_bf16(float v, float* hi, float* lo) {
    const float most = __uint_as_float(0x7f7f0000u);
    const float h = __bfloat162float(__float2bfloat16_rn(v));
    *hi = isinf(h) && !isinf(v) ? copysignf(most, v) : h;
    *lo = isfinite(*hi) ? v - *hi : 0.f;
}

// short requests, and every token's adapter; the first and the last request's CTAs also mark what lies outside
__device__ __forceinline__ void short_request(const LowJob& J, int s, int y) {
    const int warp = threadIdx.x >> 5, n_tok = (int)J.n_tok;
    if (s >= (J.n_seg > 0 ? J.n_seg : 1)) return;
    int first = 0, last = 0, a = -1;
    if (J.n_seg > 0) {
        first = min(max(J.cu_rows[s], 0), n_tok);
        last = min(max(J.cu_rows[s + 1], 0), n_tok);
        a = J.adapter_idx[s];
    }
    if (a < 0 || a >= J.n_adapters) a = -1;
    const bool later = last - first >= kShortRequest;
    if (y == 0) {
        for (int t = first + threadIdx.x; t < last; t += kLowTcThreads) J.tok_adapter[t] = a;
        if (s == 0)
            for (int t = threadIdx.x; t < first; t += kLowTcThreads) J.tok_adapter[t] = -1;
        if (s >= J.n_seg - 1)
            for (int t = last + threadIdx.x; t < n_tok; t += kLowTcThreads) J.tok_adapter[t] = -1;
    }
    if (a < 0 || later) return;
    const int cols = (J.rank + 15) / 16 * 16, row = low_row(J.rank), lo = J.rank <= 32 ? cols : row / 2;
    const int j0 = (y * kLowTcWarps + warp) * 2;
    if (j0 >= cols) return;
    for (int t = first; t < last; ++t) {
        __nv_bfloat16* v = static_cast<__nv_bfloat16*>(J.v) + (int64_t)t * row;
        low_rows<2>(J, t, a, j0, cols, [&](int c, float x) {
            float h, l;
            split_bf16(x, &h, &l);
            v[c] = __float2bfloat16_rn(h);
            v[lo + c] = __float2bfloat16_rn(l);
        });
    }
}

__global__ void __launch_bounds__(kLowTcThreads, 2)
    k_lora_wide(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap ta,
               const __grid_constant__ WideLowArgs P) {
    constexpr uint32_t COLS = 128;
    const LowJob& J = P.J;
    griddep_wait();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < J.n_zero; i += kLowTcThreads) J.zero[i] = 0;
    if ((int)blockIdx.x >= P.n_split) {  // (whole clusters; no barrier of theirs is used here)
        griddep_launch_dependents();
        const int q = (int)blockIdx.x - P.n_split;
        short_request(J, q / P.y_split, q % P.y_split);
        return;
    }
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + kLowBar);
    uint64_t* empty = full + 5;
    uint64_t* done = empty + 5;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rp = (J.rank + 15) / 16 * 16, ks = P.ks, rank = (int)(blockIdx.x % ks);
    const int stage = kXBytes + rp * kLowK * 2, S = min(5, kLowRing / stage);
    const int64_t t0 = (int64_t)(blockIdx.x / ks) * 128;
    const int kb0 = (int)((int64_t)rank * P.kb / ks), kb1 = (int)((int64_t)(rank + 1) * P.kb / ks);
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 1) tc::alloc(tslot, COLS);
    int* cu = reinterpret_cast<int*>(sm + kLowCuOff);
    const bool near_cu = J.n_seg <= kLowCu;
    if (near_cu)
        for (int i = tid; i <= J.n_seg; i += kLowTcThreads) cu[i] = J.cu_rows[i];
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    griddep_launch_dependents();
    const uint32_t tm = *tslot;
    bool ok = true;

    // the adapter of a token of a long request, else -1
    auto adapter_of = [&](int64_t t) {
        if (t >= J.n_tok) return -1;
        auto at = [&](int i) { return near_cu ? cu[i] : J.cu_rows[i]; };
        int s = -1;
        for (int hi = J.n_seg; hi - s > 1;) {  // the last s with cu_rows[s] <= t
            const int mid = (s + hi) >> 1;
            if (at(mid) <= t) s = mid;
            else hi = mid;
        }
        if (s < 0) return -1;
        const int first = max(at(s), 0), last = (int)min((int64_t)at(s + 1), J.n_tok), a = J.adapter_idx[s];
        return t >= first && t < last && last - first >= kShortRequest && a < J.n_adapters ? max(a, -1) : -1;
    };
    // those of the tile: lane l holds tokens l, l + 32, ...
    int a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = adapter_of(t0 + 32 * j + lane);
    auto next = [&](int last) {
        int m = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (a[j] > last) m = min(m, a[j]);
        return (int)__reduce_min_sync(0xffffffffu, m);
    };
    const int first = next(-1);  // the same in every warp of the cluster

    if (warp == 0) {
        uint32_t it = 0;
        for (int e = first; e != 0x7fffffff && ok; e = next(e))
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = (int)(it % S);
                ok = __all_sync(0xffffffffu, mbar_wait(empty + s, ((it / S) & 1u) ^ 1u));
                if (!ok) break;
                if (lane == 0) {
                    unsigned char* st = sm + s * stage;
                    mbar_arrive_expect_tx(full + s, (uint32_t)(kXBytes + rp * kLowK * 2));
                    tma_tile_2d(st, &tx, kb * kLowK, (int)t0, full + s);
                    tma_tile_3d(st + kXBytes, &ta, kb * kLowK, 0, e, full + s);
                }
            }
    } else if (warp == 1) {
        const uint32_t idesc = idesc_bf16(128, rp);
        uint32_t it = 0;
        for (int e = first; e != 0x7fffffff && ok; e = next(e)) {
            uint32_t off[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) off[j] = ~__ballot_sync(0xffffffffu, a[j] == e);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = (int)(it % S);
                ok = __all_sync(0xffffffffu, mbar_wait(full + s, (it / S) & 1u));
                if (!ok) break;
                tc::fence_after();
                if (lane == 0) {
                    const uint32_t a0 = tc::smem_addr(sm + s * stage), b0 = a0 + kXBytes;
#pragma unroll
                    for (int k16 = 0; k16 < kLowK / 16; ++k16)
                        mma_bf16_lanes(tm, tc::sdesc(a0 + k16 * 32), tc::sdesc(b0 + k16 * 32), idesc,
                                       kb > kb0 || k16 > 0 ? 1u : 0u, off);
                    tc::commit(empty + s);
                }
                __syncwarp();
            }
        }
        if (ok && lane == 0 && first != 0x7fffffff) tc::commit(done);  // (nobody would wait for it)
        __syncwarp();
    } else if (first != 0x7fffffff) {
        const int q4 = warp & 3;
        ok = __all_sync(0xffffffffu, mbar_wait(done, 0));
        if (ok) {
            tc::fence_after();
            float* red = reinterpret_cast<float*>(sm) + 32 * q4 + lane;  // [column][128 tokens]
            for (int c0 = 0; c0 < rp; c0 += 16) {
                float v[16];
                tc::ld16(tc::taddr(tm, 32 * q4, c0), v);
#pragma unroll
                for (int i = 0; i < 16; ++i) red[(c0 + i) * 128] = v[i];
            }
        }
    }
    tc::fence_before();
    const int bad = __syncthreads_or(!ok);
    if (bad && tid == 0) report_device_status(kDevWaitTimeout);
    if (ks > 1) {
        cluster_arrive_release();
        cluster_wait_acquire();
    }
    // this CTA's tokens, 8 columns a thread
    if (!bad && first != 0x7fffffff) {
        const int lo = J.rank <= 32 ? rp : (J.rank + 63) / 64 * 64, row = low_row(J.rank), mine = 128 / ks;
        const uint32_t own = smem_u32(sm);
        for (int i = tid; i < mine * (rp / 8); i += kLowTcThreads) {
            const int c0 = i / mine * 8, tok = rank * mine + i % mine, e = adapter_of(t0 + tok);
            if (e < 0) continue;
            float v[8] = {}, h[8], l[8];
            for (int r = 0; r < ks; ++r) {
                const uint32_t src = (ks > 1 ? mapa_shared(own, r) : own) + (uint32_t)(c0 * 128 + tok) * 4;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float p;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p) : "r"(src + j * 512) : "memory");
                    v[j] += p;
                }
            }
            const float scale = J.scale ? J.scale[e] : 1.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = c0 < J.rank ? v[j] * scale : 0.f;  // (beyond the rank 0 x, which is no 0 for an infinite x)
                split_bf16(v[j], h + j, l + j);
            }
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(J.v) + (t0 + tok) * row + c0;
            *reinterpret_cast<uint4*>(dst) = pack8(h);
            *reinterpret_cast<uint4*>(dst + lo) = pack8(l);
        }
    }
    if (ks > 1) {  // no CTA leaves while others read its shared memory
        cluster_arrive_release();
        cluster_wait_acquire();
    }
    __syncthreads();
    if (warp == 1) tc::dealloc(tm, COLS);
}

}  // namespace

cudaError_t take_device_status_lora(unsigned* out) { return take_device_status_tu(out); }

cudaError_t launch_lora_low(const LowJob& job, cudaStream_t st) {
    if (job.n_tok == 0) return cudaSuccess;
    if (!job.wide) {
        const dim3 grid((unsigned)job.n_tok, (unsigned)((job.rank + kLowWarps - 1) / kLowWarps));
        return launch_pdl(k_lora_low, grid, dim3(kLowThreads), 0, st, job);
    }
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t e = raise_smem_limit_shared(k_lora_wide, kLowSmem, smem_set);
    if (e != cudaSuccess) return e;
    CUtensorMap mx, ma;
    if (!map_rows(&mx, job.x, job.n_tok, job.k, 128) ||
        !map_stack(&ma, job.a, job.n_adapters, job.rank, job.k, (job.rank + 15) / 16 * 16))
        return cudaErrorInvalidValue;
    WideLowArgs P = {};
    P.J = job;
    P.kb = (job.k + kLowK - 1) / kLowK;
    const int64_t tiles = (job.n_tok + 127) / 128;
    P.ks = 1;
    while (P.ks < 8 && tiles * P.ks * 2 <= 2 * sm_count() && P.kb >= P.ks * 4) P.ks *= 2;
    P.n_split = (int32_t)(tiles * P.ks);
    P.y_split = ((job.rank + 15) / 16 * 16 + 2 * kLowTcWarps - 1) / (2 * kLowTcWarps);
    const int64_t shorts = (int64_t)std::max(job.n_seg, 1) * P.y_split;
    return launch_pdl_cluster(k_lora_wide, dim3((unsigned)(P.n_split + (shorts + P.ks - 1) / P.ks * P.ks)), dim3(kLowTcThreads),
                              kLowSmem, P.ks, st, mx, ma, P);
}

}  // namespace gdn
