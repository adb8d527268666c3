// gdn_few.cu -- projections of few tokens with a fused end: the gated half of a feed-forward block, a projection with
// each request's low-rank adapter beside it, and the plain projection back to the model width.
//
//   plain   out[t][n] = x_t . w_n
//   gated   out[t][n] = silu(x_t . g_n) (x_t . u_n)
//   lora    out[t][n] = x_t . w_n + v_t . b_n(adapter of t),   v_t = scale A x_t
//
// Few tokens: the weights are read once and everything else is small, so the kernel is a stream of weight tiles through
// shared memory.  A tile is 128 weight rows (gated: 64 of each matrix) and is the MMA's M side, the tokens are its N side;
// K is split over a cluster of ks CTAs whose fp32 partial products are joined through distributed shared memory, so that
// there is one launch and no workspace.
//   warp 0      TMA producer: 64-wide K blocks of the weights and the tokens into a ring of stages
//   warp 1      MMA issuer (tcgen05, bf16 operands, fp32 accumulators in TMEM)
//   warps 2..5  lora: the adapters' part of the tokens that this CTA will finish, on the CUDA cores while the weights
//               stream (a thread is an output channel; each row of b is read by one thread, once, and a token only ever
//               meets its own adapter, whatever the others hold); then accumulator -> shared memory
//   all warps   join the ks partial blocks (each CTA finishes every ks-th token), fuse, round, store
// The join adds the parts in the order of their ranks, so results do not change from call to call.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "gdn_common.cuh"
#include "gdn_gemm.cuh"
#include "gdn_internal.h"
#include "gdn_tc.cuh"
#include "gdn_tma.cuh"

namespace gdn {
namespace {

enum { kPlain = 0, kGated = 1, kLora = 2 };

constexpr int kFewThreads = 192;
constexpr int kFewM = 128;  // weight rows per tile
constexpr int kFewK = 64;   // K per stage

template <int N>
struct FewLay {
    static constexpr int W_BYTES = kFewM * kFewK * 2;
    static constexpr int X_BYTES = N * kFewK * 2;
    static constexpr int STAGE = W_BYTES + X_BYTES;
    static constexpr int STAGES = N == 16 ? 6 : N == 32 ? 5 : N == 64 ? 4 : 3;  // two CTAs on an SM
    static constexpr int RED = N * kFewM * 4;                                     // fp32 partial block, over the ring
    static constexpr int RING = STAGES * STAGE > RED ? STAGES * STAGE : RED;
    static constexpr int BAR_OFF = RING;  // full[S], empty[S], done, TMEM address
    static constexpr int ADP_OFF = BAR_OFF + (2 * STAGES + 1) * 8 + 8;
    static constexpr int SMEM_ALLOC = ADP_OFF + N * 4 + 1024;
    static_assert(2 * (SMEM_ALLOC + 1024) <= 227 * 1024, "two CTAs on an SM");
};

struct FewArgs {
    int64_t n_tok;
    int32_t n_out;    // gated: rows of each matrix
    int32_t kb;       // 64-wide K blocks
    int32_t ks;       // cluster size
    int32_t early;    // launched behind a kernel of the same call: weights may be asked for before it has ended
    __nv_bfloat16* out;
    int64_t ld;
    // lora
    const float* v;            // [n_tok][rank]
    const int32_t* tok_adapter;  // [n_tok], -1: none
    const __nv_bfloat16* b;    // [n_adapters][n_out][rank]
    int32_t rank, n_adapters;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// d[i] = v of token i . row n of its adapter's b, for the kTok tokens `tok` (adapter < 0: 0)
constexpr int kTok = 8;
__device__ __forceinline__ void adapter_part(const FewArgs& P, const int* adapter, int n, int64_t t0, int first, int step,
                                             int count, float d[kTok]) {
    const __nv_bfloat16* row[kTok];
    const float* vt[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
        d[i] = 0.f;
        const int c = first + i * step;
        const int a = i < count ? adapter[c] : -1;
        row[i] = a >= 0 && n < P.n_out ? P.b + ((int64_t)a * P.n_out + n) * P.rank : nullptr;
        vt[i] = P.v + (t0 + c) * P.rank;
    }
    for (int j = 0; j < P.rank; j += 16) {
        uint4 w[kTok][2];
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
            if (row[i]) {
                w[i][0] = *reinterpret_cast<const uint4*>(row[i] + j);
                if (j + 8 < P.rank) w[i][1] = *reinterpret_cast<const uint4*>(row[i] + j + 8);
            }
        }
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            if (!row[i]) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (j + 8 * h >= P.rank) break;
                const float4 v0 = *reinterpret_cast<const float4*>(vt[i] + j + 8 * h);
                const float4 v1 = *reinterpret_cast<const float4*>(vt[i] + j + 8 * h + 4);
                const uint32_t u[4] = {w[i][h].x, w[i][h].y, w[i][h].z, w[i][h].w};
                d[i] += __uint_as_float(u[0] << 16) * v0.x + __uint_as_float(u[0] & 0xffff0000u) * v0.y +
                        __uint_as_float(u[1] << 16) * v0.z + __uint_as_float(u[1] & 0xffff0000u) * v0.w;
                d[i] += __uint_as_float(u[2] << 16) * v1.x + __uint_as_float(u[2] & 0xffff0000u) * v1.y +
                        __uint_as_float(u[3] << 16) * v1.z + __uint_as_float(u[3] & 0xffff0000u) * v1.w;
            }
        }
    }
}

template <int N, int MODE>
__global__ void __launch_bounds__(kFewThreads, 2)
    k_few(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tw2,
          const __grid_constant__ CUtensorMap tx, const __grid_constant__ FewArgs P) {
    using L = FewLay<N>;
    constexpr int S = L::STAGES;
    // accumulator, then (lora) the adapters' part of this CTA's tokens
    constexpr uint32_t COLS = MODE == kLora ? 2 * N : (N < 32 ? 32 : N);
    // Without `early` nothing is held or asked for before everything ahead in the stream has ended.  With it, the kernel
    // ahead is one of the same call, which lets this one start only after its own wait (so all that came before it has
    // ended) and with its TMEM in hand (so holding TMEM here cannot keep it from its own).
    if (!P.early) griddep_wait();
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
    uint64_t* empty = full + S;
    uint64_t* done = empty + S;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
    int* adapter = reinterpret_cast<int*>(sm + L::ADP_OFF);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ks = P.ks, rank = (int)(blockIdx.x % ks), tile = (int)(blockIdx.x / ks);
    const int kb0 = (int)((int64_t)rank * P.kb / ks), kb1 = (int)((int64_t)(rank + 1) * P.kb / ks);
    const int64_t t0 = (int64_t)blockIdx.y * N;
    const int ncol = (int)(P.n_tok - t0 < N ? P.n_tok - t0 : N);

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 1) tc::alloc(tslot, COLS);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = *tslot;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            auto weights = [&](int kb, int s) {
                unsigned char* st = sm + s * L::STAGE;
                mbar_arrive_expect_tx(full + s, L::STAGE);
                if (MODE == kGated) {
                    tma_tile_2d(st, &tw, kb * kFewK, tile * (kFewM / 2), full + s);
                    tma_tile_2d(st + L::W_BYTES / 2, &tw2, kb * kFewK, tile * (kFewM / 2), full + s);
                } else {
                    tma_tile_2d(st, &tw, kb * kFewK, tile * kFewM, full + s);
                }
            };
            auto tokens = [&](int kb, int s) {
                tma_tile_2d(sm + s * L::STAGE + L::W_BYTES, &tx, kb * kFewK, (int)t0, full + s);
            };
            const int ahead = min(S, kb1 - kb0);
            for (int i = 0; i < ahead; ++i) weights(kb0 + i, i);
            if (P.early && MODE != kLora) griddep_wait();  // (lora: only v and the adapters come from the kernel ahead)
            for (int i = 0; i < ahead; ++i) tokens(kb0 + i, i);
            for (int i = ahead; i < kb1 - kb0; ++i) {
                const int s = i % S;
                if (!mbar_wait(empty + s, (uint32_t)(i / S - 1) & 1u)) {
                    ok = false;
                    break;
                }
                weights(kb0 + i, s);
                tokens(kb0 + i, s);
            }
        } else if (P.early && MODE != kLora) {
            griddep_wait();
        }
    } else if (warp == 1) {
        if (P.early && MODE != kLora) griddep_wait();
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16(kFewM, N);
            for (int i = 0; i < kb1 - kb0; ++i) {
                const int s = i % S;
                if (!mbar_wait(full + s, (uint32_t)(i / S) & 1u)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint32_t a0 = tc::smem_addr(sm + s * L::STAGE), b0 = a0 + L::W_BYTES;
#pragma unroll
                for (int k16 = 0; k16 < kFewK / 16; ++k16)
                    mma_bf16(tm, tc::sdesc(a0 + k16 * 32), tc::sdesc(b0 + k16 * 32), idesc, i > 0 || k16 > 0 ? 1u : 0u);
                tc::commit(empty + s);
            }
            if (ok) tc::commit(done);
        }
    } else {
        if (P.early) griddep_wait();
        griddep_launch_dependents();
        const int q4 = warp & 3;  // TMEM lanes 32 q4 .. are this warp's
        const int row = 32 * q4 + lane;
        const int mine = ncol > rank ? (ncol - rank + ks - 1) / ks : 0;  // tokens rank, rank + ks, ... are finished here
        if (MODE == kLora) {
            for (int c = tid - 64; c < N; c += 128) {
                const int a = c < ncol ? P.tok_adapter[t0 + c] : -1;
                adapter[c] = a < P.n_adapters ? a : -1;
            }
            named_bar_sync(1, 128);
            for (int i0 = 0; i0 < mine; i0 += 2 * kTok) {
                float d[2 * kTok];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    adapter_part(P, adapter, tile * kFewM + row, t0, rank + (i0 + h * kTok) * ks, ks,
                                 mine - i0 - h * kTok, d + h * kTok);
                tc::st16(tc::taddr(tm, 32 * q4, N + i0), d);
            }
        }
        const bool w = mbar_wait(done, 0);
        ok = w;
        if (__all_sync(0xffffffffu, w)) {
            tc::fence_after();
            // every MMA has read its operands: the ring's memory takes the partial block, [token][128 rows]
            float* red = reinterpret_cast<float*>(sm) + row;
            for (int c0 = 0; c0 < ncol; c0 += 16) {
                float v[16];
                tc::ld16(tc::taddr(tm, 32 * q4, c0), v);
#pragma unroll
                for (int c = 0; c < 16; ++c) red[(c0 + c) * kFewM] = v[c];
            }
            if (MODE == kLora)
                for (int i0 = 0; i0 < mine; i0 += 16) {
                    float v[16];
                    tc::ld16(tc::taddr(tm, 32 * q4, N + i0), v);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i0 + i < mine) red[(rank + (i0 + i) * ks) * kFewM] += v[i];
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
    // a thread takes 4 rows of a token: 32 lanes are the 128 rows (gated: 16 lanes, each with both matrices' rows)
    if (!bad) {
        constexpr int LPT = MODE == kGated ? 16 : 32;
        constexpr int ROWS = MODE == kGated ? kFewM / 2 : kFewM;
        const int n = tile * ROWS + 4 * (tid % LPT);
        const uint32_t own = smem_u32(sm) + 16 * (tid % LPT);
        const bool vec = n + 4 <= P.n_out && (P.ld & 3) == 0 && (reinterpret_cast<uintptr_t>(P.out) & 7) == 0;
        for (int i = tid / LPT;; i += kFewThreads / LPT) {
            const int c = rank + i * ks;
            if (c >= ncol) break;
            float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
            for (int r = 0; r < ks; ++r) {
                const uint32_t a = (ks > 1 ? mapa_shared(own, r) : own) + c * (kFewM * 4);
                const float4 p = ks > 1 ? ld_cluster_f4(a) : *reinterpret_cast<const float4*>(sm + (a - smem_u32(sm)));
                g.x += p.x, g.y += p.y, g.z += p.z, g.w += p.w;
                if (MODE == kGated) {
                    const float4 q = ks > 1 ? ld_cluster_f4(a + kFewM * 2)
                                            : *reinterpret_cast<const float4*>(sm + (a - smem_u32(sm)) + kFewM * 2);
                    u.x += q.x, u.y += q.y, u.z += q.z, u.w += q.w;
                }
            }
            float o[4] = {g.x, g.y, g.z, g.w};
            if (MODE == kGated) {
                o[0] = siluf_(g.x) * u.x, o[1] = siluf_(g.y) * u.y, o[2] = siluf_(g.z) * u.z, o[3] = siluf_(g.w) * u.w;
            }
            __nv_bfloat16* dst = P.out + (t0 + c) * P.ld + n;
            if (vec) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(o[0], o[1]), hi = __floats2bfloat162_rn(o[2], o[3]);
                *reinterpret_cast<uint2*>(dst) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < P.n_out) dst[e] = __float2bfloat16_rn(o[e]);
            }
        }
    }
    if (ks > 1) {  // no CTA leaves while others read its shared memory
        cluster_arrive_release();
        cluster_wait_acquire();
    }
    __syncthreads();
    if (warp == 1) tc::dealloc(tm, COLS);
}

template <int N, int MODE>
cudaError_t launch_few_n(const FewJob& job, int ks, cudaStream_t st) {
    using L = FewLay<N>;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = raise_smem_limit(k_few<N, MODE>, L::SMEM_ALLOC, smem_set);
    if (e != cudaSuccess) return e;
    constexpr int rows = MODE == kGated ? kFewM / 2 : kFewM;
    CUtensorMap mw, mw2, mx;
    if (!map_rows(&mw, job.w, job.n_out, job.k, rows) || !map_rows(&mw2, job.w2 ? job.w2 : job.w, job.n_out, job.k, rows) ||
        !map_rows(&mx, job.x, job.n_tok, job.k, N))
        return cudaErrorInvalidValue;
    FewArgs P = {};
    P.n_tok = job.n_tok;
    P.n_out = job.n_out;
    P.kb = (job.k + kFewK - 1) / kFewK;
    P.ks = ks;
    P.early = job.early;
    P.out = static_cast<__nv_bfloat16*>(job.out);
    P.ld = job.ld;
    P.v = job.v;
    P.tok_adapter = job.tok_adapter;
    P.b = static_cast<const __nv_bfloat16*>(job.b);
    P.rank = job.rank;
    P.n_adapters = job.n_adapters;
    const unsigned tiles = (unsigned)((job.n_out + rows - 1) / rows);
    return launch_pdl_cluster(k_few<N, MODE>, dim3(tiles * ks, (unsigned)((job.n_tok + N - 1) / N)), dim3(kFewThreads),
                              L::SMEM_ALLOC, ks, st, mw, mw2, mx, P);
}

// Cluster size: the CTAs run in waves of two per SM, and a CTA costs its K blocks and a start and end worth about
// kFewEnds of them.
constexpr int kFewEnds = 6;
int few_split(int64_t tiles, int kb) {
    const int64_t slots = 2 * (int64_t)sm_count();
    int best = 1;
    int64_t least = -1;
    for (int ks = 1; ks <= 8 && ks <= std::max(1, kb / 2); ++ks) {
        const int64_t cost = (tiles * ks + slots - 1) / slots * ((kb + ks - 1) / ks + kFewEnds);
        if (least < 0 || cost < least) {
            least = cost;
            best = ks;
        }
    }
    return best;
}

template <int MODE>
cudaError_t launch_few_mode(const FewJob& job, cudaStream_t st) {
    constexpr int rows = MODE == kGated ? kFewM / 2 : kFewM;
    const int N = job.n_tok <= 16 ? 16 : job.n_tok <= 32 ? 32 : job.n_tok <= 64 ? 64 : 128;
    const int64_t tiles = (job.n_out + rows - 1) / rows * ((job.n_tok + N - 1) / N);
    const int ks = few_split(tiles, (job.k + kFewK - 1) / kFewK);
    switch (N) {
        case 16: return launch_few_n<16, MODE>(job, ks, st);
        case 32: return launch_few_n<32, MODE>(job, ks, st);
        case 64: return launch_few_n<64, MODE>(job, ks, st);
        default: return launch_few_n<128, MODE>(job, ks, st);
    }
}

}  // namespace

cudaError_t take_device_status_few(unsigned* out) { return take_device_status_tu(out); }

cudaError_t launch_few(const FewJob& job, cudaStream_t st) {
    if (job.n_tok == 0 || job.n_out == 0) return cudaSuccess;
    return job.rank > 0 ? launch_few_mode<kLora>(job, st)
                        : job.w2 ? launch_few_mode<kGated>(job, st) : launch_few_mode<kPlain>(job, st);
}

}  // namespace gdn
