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
//   warps 2..5  accumulator -> shared memory; lora: before that, while the weights stream, the adapters' part of the
//               tokens that this CTA will finish, on the CUDA cores (a thread is an output channel; each row of b meets
//               one token once, and a token only its own adapter, whatever the others hold)
//   warp 6      lora: the 128 rows of b of each such token, and its v, into a second ring of shared memory.  Bulk copies: the
//               rows of a token lie together, and while the weights saturate the memory a load takes 3 us, so that threads
//               which load, use and load again cannot keep up (64 requests: 40 us that way)
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

constexpr int kFewM = 128;  // weight rows per tile
constexpr int kFewK = 64;   // K per stage
constexpr int kFewAhead = 3;  // stages of weights asked for before the kernel ahead has ended
template <int MODE>
constexpr int few_threads() { return MODE == kLora ? 224 : 192; }

// Two CTAs on an SM.  What they have in flight covers the memory's latency several times over; more of it only makes
// every other load wait longer, so the weights' ring is the smaller one where the rows of b stream beside them.
constexpr int kRowSlots = 16;  // lora: tokens in the ring of adapter rows, at most
constexpr int few_stage(int n) { return (kFewM + n) * kFewK * 2; }
constexpr int few_lora_stages(int n) { return n <= 32 ? 3 : 2; }
constexpr int few_row_ring(int n) { return 108 * 1024 - few_lora_stages(n) * few_stage(n); }
constexpr int few_row_slot(int rank) { return kFewM * rank * 2 + rank * 4; }  // 128 rows of b, then v
template <int N, int MODE>
struct FewLay {
    static constexpr int W_BYTES = kFewM * kFewK * 2;
    static constexpr int STAGE = few_stage(N);
    static constexpr int STAGES = MODE == kLora ? few_lora_stages(N) : N == 16 ? 6 : N == 32 ? 5 : N == 64 ? 4 : 3;
    static constexpr int RING = STAGES * STAGE;  // the fp32 partial block lies over it at the end
    static constexpr int ROW_OFF = RING;
    static constexpr int ROW_RING = MODE == kLora ? few_row_ring(N) : 0;
    // full[S], empty[S], done, row_full[], row_empty[], TMEM address, the tokens' adapters
    static constexpr int BAR_OFF = ROW_OFF + ROW_RING;
    static constexpr int ADP_OFF = BAR_OFF + (2 * STAGES + 1 + (MODE == kLora ? 2 * kRowSlots : 0)) * 8 + 8;
    static constexpr int SMEM_ALLOC = ADP_OFF + (MODE == kLora ? N * 4 : 0) + 1024;
    static_assert(RING >= N * kFewM * 4, "the partial block");
    static_assert(MODE != kLora || ROW_RING >= few_row_slot(128), "a token of the largest rank");
    static_assert(2 * (SMEM_ALLOC + 1024) <= 227 * 1024, "CTAs on an SM");
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
    const int32_t *cu_rows, *adapter_idx;
    const __nv_bfloat16* b;    // [n_adapters][n_out][rank]
    int32_t rank, n_adapters, n_seg;
    int32_t* zero;  // counters of a kernel behind this one, set to zero here
    int32_t n_zero;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_tmem1(uint32_t taddr, float v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v)) : "memory");
}

__device__ __forceinline__ void named_bar_arrive(int id, int count) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// one row of b (bf16, in shared memory, 16 bytes `pieces` to a row) . v (fp32, in shared memory).  The lanes start at
// different pieces, so that 8 of them reach all banks whatever the rows' length.
__device__ __forceinline__ float row_dot(const unsigned char* rows, int row, const float* v, int pieces, int start) {
    const uint4* b = reinterpret_cast<const uint4*>(rows) + row * pieces;
    float d = 0.f;
    int c = start;
    for (int j = 0; j < pieces; ++j) {
        const uint4 w = b[c];
        const float4 v0 = reinterpret_cast<const float4*>(v)[2 * c], v1 = reinterpret_cast<const float4*>(v)[2 * c + 1];
        d = fmaf(__uint_as_float(w.x << 16), v0.x, d);
        d = fmaf(__uint_as_float(w.x & 0xffff0000u), v0.y, d);
        d = fmaf(__uint_as_float(w.y << 16), v0.z, d);
        d = fmaf(__uint_as_float(w.y & 0xffff0000u), v0.w, d);
        d = fmaf(__uint_as_float(w.z << 16), v1.x, d);
        d = fmaf(__uint_as_float(w.z & 0xffff0000u), v1.y, d);
        d = fmaf(__uint_as_float(w.w << 16), v1.z, d);
        d = fmaf(__uint_as_float(w.w & 0xffff0000u), v1.w, d);
        if (++c == pieces) c = 0;
    }
    return d;
}

template <int N, int MODE>
__global__ void __launch_bounds__(few_threads<MODE>(), 2)
    k_few(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tw2,
          const __grid_constant__ CUtensorMap tx, const __grid_constant__ FewArgs P) {
    using L = FewLay<N, MODE>;
    constexpr int S = L::STAGES, THREADS = few_threads<MODE>();
    // accumulator, then (lora) the adapters' part of this CTA's tokens
    constexpr uint32_t COLS = MODE == kLora ? 2 * N : (N < 32 ? 32 : N);
    // Without `early` nothing is held or asked for before everything ahead in the stream has ended.  With it, the kernel
    // ahead is one of the same call, which lets this one start only after its own wait (so all that came before it has
    // ended) and with its TMEM in hand (so holding TMEM here cannot keep it from its own).
    if (!P.early) griddep_wait();
    if (P.n_zero > 0 && blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < P.n_zero; i += few_threads<MODE>()) P.zero[i] = 0;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
    uint64_t* empty = full + S;
    uint64_t* done = empty + S;
    uint64_t* row_full = done + 1;
    uint64_t* row_empty = row_full + kRowSlots;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(MODE == kLora ? row_empty + kRowSlots : done + 1);
    int* adapter = reinterpret_cast<int*>(sm + L::ADP_OFF);  // of the tokens that this CTA finishes
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ks = P.ks, rank = (int)(blockIdx.x % ks), tile = (int)(blockIdx.x / ks);
    const int kb0 = (int)((int64_t)rank * P.kb / ks), kb1 = (int)((int64_t)(rank + 1) * P.kb / ks);
    const int64_t t0 = (int64_t)blockIdx.y * N;
    const int ncol = (int)(P.n_tok - t0 < N ? P.n_tok - t0 : N);
    const int mine = ncol > rank ? (ncol - rank + ks - 1) / ks : 0;  // tokens rank, rank + ks, ... are finished here
    const int slot_bytes = few_row_slot(P.rank);  // in the ring of adapter rows
    const int slots = MODE == kLora ? min(kRowSlots, L::ROW_RING / slot_bytes) : 1;

    if (tid == 0) {
        if (MODE == kLora)
            for (int s = 0; s < slots; ++s) {
                mbar_init(row_full + s, 1);
                mbar_init(row_empty + s, 4);
            }
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
            // weights ahead of the wait, but not the whole ring of them: the tokens of the first stage come behind
            const int ahead = min(S, kb1 - kb0), early = P.early && MODE != kLora ? min(kFewAhead, ahead) : 0;
            for (int i = 0; i < early; ++i) weights(kb0 + i, i);
            if (P.early && MODE != kLora) griddep_wait();  // (lora: only v and the adapters come from the kernel ahead)
            for (int i = 0; i < ahead; ++i) {
                if (i >= early) weights(kb0 + i, i);
                tokens(kb0 + i, i);
            }
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
    } else if (MODE == kLora && warp == 6) {
        // The adapters of a decoding batch (request t is token t) are known without the kernel ahead, and with them the rows
        // of b; only v has to be waited for.
        int a[(N + 31) / 32];
        bool known = true;
#pragma unroll
        for (int j = 0; j < (N + 31) / 32; ++j) {
            const int i = 32 * j + lane;
            const int t = (int)t0 + rank + i * ks;
            a[j] = -1;
            if (i < mine) {
                known = known && t < P.n_seg && P.cu_rows[t] <= t && t < P.cu_rows[t + 1];
                if (t < P.n_seg) a[j] = P.adapter_idx[t];
            }
        }
        known = __all_sync(0xffffffffu, known);
        if (!known) griddep_wait();
#pragma unroll
        for (int j = 0; j < (N + 31) / 32; ++j) {
            const int i = 32 * j + lane;
            if (i >= mine) continue;
            if (!known) a[j] = P.tok_adapter[t0 + rank + i * ks];
            adapter[i] = a[j] >= 0 && a[j] < P.n_adapters ? a[j] : -1;
        }
        __syncwarp();
        named_bar_arrive(1, 160);
        if (lane == 0) {
            const int rows = min(kFewM, P.n_out - tile * kFewM);
            const uint32_t b_bytes = (uint32_t)rows * P.rank * 2, v_bytes = (uint32_t)P.rank * 4;
            auto slot_of = [&](int k) { return sm + L::ROW_OFF + (k % slots) * slot_bytes; };
            auto copy_b = [&](int i, int k) {
                mbar_arrive_expect_tx(row_full + k % slots, b_bytes + v_bytes);
                bulk_g2s(slot_of(k), P.b + ((int64_t)adapter[i] * P.n_out + tile * kFewM) * P.rank, b_bytes,
                         row_full + k % slots);
            };
            auto copy_v = [&](int i, int k) {
                bulk_g2s(slot_of(k) + kFewM * P.rank * 2, P.v + (t0 + rank + (int64_t)i * ks) * P.rank, v_bytes,
                         row_full + k % slots);
            };
            int i = 0, k = 0, i_v = 0, k_v = 0;
            for (; i < mine && k < slots; ++i)
                if (adapter[i] >= 0) copy_b(i, k++);
            griddep_wait();
            for (; i_v < i; ++i_v)
                if (adapter[i_v] >= 0) copy_v(i_v, k_v++);
            for (; i < mine; ++i) {
                if (adapter[i] < 0) continue;
                if (!mbar_wait(row_empty + k % slots, (uint32_t)(k / slots - 1) & 1u)) {
                    ok = false;
                    break;
                }
                copy_b(i, k);
                copy_v(i, k++);
            }
        }
        __syncwarp();
    } else {
        if (P.early) griddep_wait();
        griddep_launch_dependents();
        const int q4 = warp & 3;  // TMEM lanes 32 q4 .. are this warp's
        const int row = 32 * q4 + lane;
        if (MODE == kLora) {
            named_bar_sync(1, 160);
            const int pieces = P.rank / 8, shift = pieces & 1 ? 3 : pieces & 2 ? 2 : pieces & 4 ? 1 : 0;
            const int start = (lane >> shift) % pieces;
            int k = 0;
            for (int i = 0; i < mine && ok; ++i) {
                float d = 0.f;
                if (adapter[i] >= 0) {
                    const int s = k % slots;
                    ok = __all_sync(0xffffffffu, mbar_wait(row_full + s, (uint32_t)(k / slots) & 1u));
                    const unsigned char* st = sm + L::ROW_OFF + s * slot_bytes;
                    if (ok) d = row_dot(st, row, reinterpret_cast<const float*>(st + kFewM * P.rank * 2), pieces, start);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(row_empty + s);
                    ++k;
                }
                st_tmem1(tc::taddr(tm, 32 * q4, N + i), d);
            }
            tc::st_wait();
        }
        ok = __all_sync(0xffffffffu, mbar_wait(done, 0)) && ok;
        if (ok) {
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
    // A thread takes 4 rows of a token: 32 lanes are the 128 rows (gated: 16 lanes, each with both matrices' rows).  The reads
    // from four CTAs are under way together.
    constexpr int LPT = MODE == kGated ? 16 : 32;
    constexpr int ROWS = MODE == kGated ? kFewM / 2 : kFewM;
    const int n = tile * ROWS + 4 * (tid % LPT);
    const uint32_t own = smem_u32(sm) + 16 * (tid % LPT);
    const bool vec = n + 4 <= P.n_out && (P.ld & 3) == 0 && (reinterpret_cast<uintptr_t>(P.out) & 7) == 0;
    for (int i = tid / LPT; i < mine && !bad; i += THREADS / LPT) {
        const int c = rank + i * ks;
        float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
#pragma unroll 4
        for (int r = 0; r < ks; ++r) {
            const uint32_t at = (ks > 1 ? mapa_shared(own, r) : own) + c * (kFewM * 4);
            const float4 p = ld_cluster_f4(at);
            g.x += p.x, g.y += p.y, g.z += p.z, g.w += p.w;
            if (MODE == kGated) {
                const float4 q = ld_cluster_f4(at + kFewM * 2);
                u.x += q.x, u.y += q.y, u.z += q.z, u.w += q.w;
            }
        }
        float o[4] = {g.x, g.y, g.z, g.w};
        if (MODE == kGated) {
            o[0] = silu_gate(g.x) * u.x, o[1] = silu_gate(g.y) * u.y, o[2] = silu_gate(g.z) * u.z, o[3] = silu_gate(g.w) * u.w;
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
    __syncwarp();
    if (warp == 1) tc::dealloc(tm, COLS);
    if (ks > 1) {  // no CTA leaves while others read its shared memory
        cluster_arrive_release();
        cluster_wait_acquire();
    }
}

template <int N, int MODE>
cudaError_t launch_few_n(const FewJob& job, int ks, cudaStream_t st) {
    using L = FewLay<N, MODE>;
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t e = raise_smem_limit_shared(k_few<N, MODE>, L::SMEM_ALLOC, smem_set);
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
    P.early = job.early;
    P.out = static_cast<__nv_bfloat16*>(job.out);
    P.ld = job.ld;
    P.v = job.v;
    P.tok_adapter = job.tok_adapter;
    P.b = static_cast<const __nv_bfloat16*>(job.b);
    P.rank = job.rank;
    P.n_adapters = job.n_adapters;
    P.n_seg = job.n_seg;
    P.zero = job.zero;
    P.n_zero = job.n_zero;
    P.cu_rows = job.cu_rows;
    P.adapter_idx = job.adapter_idx;
    const unsigned tiles = (unsigned)((job.n_out + rows - 1) / rows);
    P.ks = ks;
    return launch_pdl_cluster(k_few<N, MODE>, dim3(tiles * ks, (unsigned)((job.n_tok + N - 1) / N)), dim3(few_threads<MODE>()),
                              L::SMEM_ALLOC, ks, st, mw, mw2, mx, P);
}

template <int MODE>
cudaError_t launch_few_mode(const FewJob& job, const FewPlan& plan, cudaStream_t st) {
    switch (plan.n) {
        case 16: return launch_few_n<16, MODE>(job, plan.ks, st);
        case 32: return launch_few_n<32, MODE>(job, plan.ks, st);
        case 64: return launch_few_n<64, MODE>(job, plan.ks, st);
        default: return launch_few_n<128, MODE>(job, plan.ks, st);
    }
}

}  // namespace

cudaError_t take_device_status_few(unsigned* out) { return take_device_status_tu(out); }

// Tokens of a tile and cluster size.  The CTAs run in waves, and a CTA costs its K blocks (0.3 us each, more with more
// tokens), a start and an end, a little for each CTA of its cluster, and with adapters its share of the tokens (0.3 us each at
// rank 16, 0.7 at 64).  `us100` was 0.65 to 1.2 of the time measured at 65 to 1500 tokens without adapters (fewer tokens:
// 0.5 to 0.9, bound by the weights' bytes, which are not counted), 0.6 to 1.5 with them at 1 to 1500 tokens and ranks 16 to 128.
// A tile takes the fewest tokens that hold all of them, 128 at most; with adapters also fewer, where more CTAs then share
// the tokens at the price of reading the weights again.  Depends on the sizes only.
FewPlan few_plan(int64_t n_tok, int32_t n_out, int32_t k, bool gated, int32_t rank) {
    static_assert(kProjTokens / 128 <= 65535, "tiles of 128 tokens in the grid's y");
    // CTAs of clusters of 1 .. 8 that run at the same time on 152 SMs, two on each: clusters of 3, 5 and more leave some of a
    // GPC's SMs empty (cudaOccupancyMaxActiveClusters)
    constexpr int kSlots[9] = {0, 304, 304, 276, 288, 280, 276, 210, 240};
    const int rows = gated ? kFewM / 2 : kFewM, kb = (k + kFewK - 1) / kFewK;
    const int most = n_tok <= 16 ? 16 : n_tok <= 32 ? 32 : n_tok <= 64 ? 64 : 128;
    FewPlan plan{most, 1, -1};
    for (int n = most; n >= (rank > 0 ? 16 : most); n /= 2) {
        const int64_t tiles_t = (n_tok + n - 1) / n, tiles = (n_out + rows - 1) / rows * tiles_t;
        // a token's rows of b; where the ring holds those of one token only, nothing is under way while they are used
        const int per_tok = rank > 0 ? 6 + rank / 4 + (few_row_ring(n) < 2 * few_row_slot(rank) ? 36 : 0) : 0;
        if (tiles_t > 65535) break;  // the grid's limit, which the first of these tiles stays within
        for (int c = 1; c <= 8 && c <= std::max(1, kb / 2); ++c) {
            const int64_t tok = (std::min<int64_t>(n, n_tok) + c - 1) / c;
            const int64_t one = (kb + c - 1) / c * 10 * (128 + n) / 128 + 80 + 10 * c + tok * per_tok;
            const int64_t cost = 3 * ((tiles * c + kSlots[c] - 1) / kSlots[c]) * one;
            if (plan.us100 < 0 || cost < plan.us100) plan = {n, c, cost};
        }
    }
    return plan;
}

cudaError_t launch_few(const FewJob& job, cudaStream_t st) {
    if (job.n_tok == 0 || job.n_out == 0) return cudaSuccess;
    const FewPlan plan = few_plan(job.n_tok, job.n_out, job.k, job.w2 != nullptr, job.rank);
    return job.rank > 0 ? launch_few_mode<kLora>(job, plan, st)
                        : job.w2 ? launch_few_mode<kGated>(job, plan, st) : launch_few_mode<kPlain>(job, plan, st);
}

}  // namespace gdn
