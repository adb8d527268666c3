// gdn_wide.cu -- projections of many tokens with a fused end (the same three as gdn_few.cu: plain, gated, lora), on
// pairs of SMs.
//
// A tile is 256 tokens x 256 accumulator columns.  The two CTAs of a cluster make it together (tcgen05 cta_group::2): each
// holds 128 of the tokens (its TMEM lanes) and loads half of the weight rows, which the MMA reads from both shared
// memories, so that a weight row is fetched once per 256 tokens and each SM's shared memory is read at half the rate
// of two tiles on their own.
//   warp 0      TMA producer (each CTA its own halves; both halves' bytes are counted on the first CTA's barrier)
//   warp 1      MMA issuer (the first CTA's; it commits to both CTAs' barriers)
//   warps 2..5  epilogue: accumulator -> registers -> bf16 -> shared memory -> TMA store, a token a thread; the other
//               half of TMEM takes the next tile meanwhile
// gated: the first CTA loads rows of w_gate and the second the same rows of w_up, so that columns c and c + 128 of
// the accumulator are a gate and its value, in one thread.
// lora: after the K blocks of x and w come, for each adapter that the tile's tokens use, its rows of b against the low-rank
// activations v, which stay in shared memory for the tile.  The MMA leaves the lanes of all other tokens as they are (its lane mask), so
// a tile may hold any mix of requests and a token meets its own adapter only, whatever the others hold.  v is carried as two bf16
// numbers, v = hi + lo to 2^-16, in place of one rounding to 2^-8 that the delta of a strong adapter would show.
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

constexpr int kWideThreads = 192;
constexpr int kWideTok = 256;  // tokens of a pair
constexpr int kWideK = 64;     // K per stage
constexpr int kHalfBytes = 128 * kWideK * 2;        // 128 rows of x, or (at most) of the weights
constexpr int kStageBytes = 2 * kHalfBytes;
constexpr int kStoreBytes = 32 * 128;  // 32 tokens x 64 columns; two per epilogue warp
// Stages of a pair's ring.  lora gives up one of them, or two above 64 ranks, for the tile's v.
constexpr int wide_stages(bool lora, int rank) { return !lora ? 6 : rank <= 64 ? 5 : 4; }
constexpr int kVOff = 5 * kStageBytes;          // v: blocks of 128 tokens x 64 (rank above 64: four, from 4 stages on)
constexpr int kStoreOff = 6 * kStageBytes;
constexpr int kBarOff = kStoreOff + 8 * kStoreBytes;  // full[6], empty[6], acc_full[2], acc_empty[2], v_full, v_empty, TMEM address
constexpr int kWideSmem = kBarOff + (2 * 6 + 6) * 8 + 16 + 1024;
static_assert(kWideSmem <= 227 * 1024, "shared memory of a CTA");
constexpr int64_t kPartFloats = 128 * 256;  // a CTA's accumulator of one part of a tile

struct WideArgs {
    int64_t n_tok, n_tiles;
    int32_t n_out;
    int32_t kb;          // 64-wide K blocks
    // Tiles from n_whole on, which would leave pairs idle in a last wave of their own, are split along K: job n_whole + i is
    // part i % split of tile n_whole + i / split.
    int64_t n_whole;
    int32_t split;
    float* part;       // [split tile][part][CTA of the pair][64 groups of 4 columns][128 tokens][4]
    int32_t* arrived;  // [split tile][CTA][epilogue warp], zero at the start
    int32_t tiles_n, tiles_t;
    int32_t token_fast;  // tile order: token blocks fastest (1) or weight blocks fastest (0)
    int32_t n_full;      // columns that go by TMA: n_out rounded down to 16 bytes
    __nv_bfloat16* out;  // the others
    int64_t ld;
    int32_t* zero;  // counters of the kernel behind this one, set to zero here
    int32_t n_zero;
    // lora
    const int32_t* tok_adapter;
    int32_t rank, n_adapters;
};

__device__ __forceinline__ void mma2_bf16(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
        : "memory");
}

// adds onto the accumulator in the lanes whose bit in `off` is clear (words 0..3: the first CTA's 128 lanes)
__device__ __forceinline__ void mma2_bf16_lanes(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, const uint32_t off[8]) {
    asm volatile(
        "{\n .reg .pred p;\n setp.eq.b32 p, 0, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7, %8, %9, %10, %11}, p;\n}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]), "r"(off[4]), "r"(off[5]),
        "r"(off[6]), "r"(off[7])
        : "memory");
}

// all earlier MMAs of this thread done -> an arrival on the barrier at this offset in both CTAs
__device__ __forceinline__ void commit2(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// loads into this CTA's shared memory that are counted on a barrier of either CTA of the pair
__device__ __forceinline__ void tma2_2d(void* dst, const void* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma2_3d(void* dst, const void* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_store_2d(const void* map, int x, int y, const void* src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
                 "r"(smem_u32(src))
                 : "memory");
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void alloc2(uint32_t* slot, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc2(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// What a job covers.  The smaller operand goes fastest, it is the one that every sweep reads again.
struct Tile {
    int tt, wn;        // token block, weight block
    int kb0, kb1;      // K blocks
    int at, part;      // split tile (-1: whole) and part
    bool last;         // the part that takes the adapters
};
__device__ __forceinline__ Tile wide_tile(const WideArgs& P, int64_t job) {
    Tile T;
    int64_t tile = job;
    T.at = -1, T.part = 0, T.kb0 = 0, T.kb1 = P.kb;
    if (job >= P.n_whole && P.split > 1) {
        T.at = (int)((job - P.n_whole) / P.split);
        T.part = (int)((job - P.n_whole) % P.split);
        T.kb0 = (int)((int64_t)T.part * P.kb / P.split);
        T.kb1 = (int)((int64_t)(T.part + 1) * P.kb / P.split);
        tile = P.n_whole + T.at;
    }
    T.last = T.kb1 == P.kb;
    if (P.token_fast) {
        T.wn = (int)(tile / P.tiles_t);
        T.tt = (int)(tile % P.tiles_t);
    } else {
        T.wn = (int)(tile % P.tiles_n);
        T.tt = (int)(tile / P.tiles_n);
    }
    return T;
}

constexpr int kNoMore = 0x7fffffff;

// The adapters that a tile's 256 tokens use, by a whole warp: lane l holds those of tokens l, l + 32, ...
struct TileAdapters {
    int a[8], last;
    __device__ __forceinline__ void load(const WideArgs& P, int tt, int lane) {
        last = -1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t t = (int64_t)tt * kWideTok + 32 * j + lane;
            const int v = t < P.n_tok ? P.tok_adapter[t] : -1;
            a[j] = v >= 0 && v < P.n_adapters ? v : -1;
        }
    }
    // the next one in ascending order
    __device__ __forceinline__ int next() {
        int m = kNoMore;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (a[j] > last) m = min(m, a[j]);
        last = __reduce_min_sync(0xffffffffu, m);
        return last;
    }
};

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
    k_wide(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw,
           const __grid_constant__ CUtensorMap tw2, const __grid_constant__ CUtensorMap tout,
           const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tb, const __grid_constant__ WideArgs P) {
    const int S = wide_stages(MODE == kLora, P.rank);
    // lora: behind the kernel that makes v, which lets this one start only after its own wait and with its TMEM in hand: x and
    // the weights are there, only v, the adapters and the counters have to be waited for.  Else nothing is held or asked for
    // while kernels ahead still run.
    constexpr bool kEarly = MODE == kLora;
    if (!kEarly) griddep_wait();
    if (!kEarly && blockIdx.x == 0)
        for (int i = threadIdx.x; i < P.n_zero; i += kWideThreads) P.zero[i] = 0;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + kBarOff);
    uint64_t* empty = full + 6;
    uint64_t* acc_full = empty + 6;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* v_full = acc_empty + 2;
    uint64_t* v_empty = v_full + 1;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(v_empty + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = (int)(blockIdx.x & 1);
    const int64_t tile0 = blockIdx.x >> 1, tstep = gridDim.x >> 1;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full + b, 1);
            mbar_init(acc_empty + b, 8);  // the epilogue warps of both CTAs
        }
        mbar_init(v_full, 1);
        mbar_init(v_empty, 1);
        fence_mbar_init();
    }
    if (warp == 1) alloc2(tslot, 512);
    tc::fence_before();
    __syncthreads();
    cluster_arrive_release();  // the other CTA's barriers and TMEM are ready
    cluster_wait_acquire();
    tc::fence_after();
    if (!kEarly) griddep_launch_dependents();
    const uint32_t tm = *tslot;
    bool ok = true;

    // lora: v of a tile is vb blocks of 64 columns, [hi | lo] in one up to 32 ranks, else those of hi, then those of lo; an
    // adapter's rows of b are bb blocks
    const int rp = (P.rank + 15) / 16, bb = (P.rank + 63) / 64, vb = P.rank <= 32 ? 1 : 2 * bb;
    unsigned char* vs = sm + (P.rank <= 64 ? kVOff : kVOff - kStageBytes);
    uint32_t st_i = 0, st_ph = 0;  // stage and its use's parity
    auto next_stage = [&] {
        if (++st_i == (uint32_t)S) {
            st_i = 0;
            st_ph ^= 1u;
        }
    };

    if (warp == 0) {
        uint32_t n_v = 0;
        // waits for the stage's turn; the first CTA's barrier expects both CTAs' bytes
        auto turn = [&](int bytes) {
            const bool w = mbar_wait(empty + st_i, st_ph ^ 1u);
            ok = __all_sync(0xffffffffu, w);
            if (ok && cta == 0 && lane == 0) mbar_arrive_expect_tx(full + st_i, 2u * (uint32_t)bytes);
        };
        for (int64_t tile = tile0; tile < P.n_tiles && ok; tile += tstep) {
            const Tile T = wide_tile(P, tile);
            const int row = T.tt * kWideTok + 128 * cta, wrow = MODE == kGated ? T.wn * 128 : T.wn * 256 + 128 * cta;
            const void* wmap = MODE == kGated && cta == 1 ? &tw2 : &tw;
            TileAdapters ta;
            if (MODE == kLora && tile != tile0) ta.load(P, T.tt, lane);
            for (int kb = T.kb0; kb < T.kb1 && ok; ++kb, next_stage()) {
                turn(2 * kHalfBytes);
                if (ok && lane == 0) {
                    unsigned char* st = sm + st_i * kStageBytes;
                    const uint32_t bar = mapa_shared(smem_u32(full + st_i), 0);
                    tma2_2d(st, &tx, kb * kWideK, row, bar);
                    tma2_2d(st + kHalfBytes, wmap, kb * kWideK, wrow, bar);
                }
            }
            if (MODE == kLora && tile == tile0) {
                griddep_wait();
                ta.load(P, T.tt, lane);
            }
            if (MODE == kLora && ok && T.last) {
                int a = ta.next();
                if (a == kNoMore) continue;
                const bool w = mbar_wait(v_empty, (n_v & 1u) ^ 1u);
                ok = __all_sync(0xffffffffu, w);
                ++n_v;
                if (!ok) break;
                if (lane == 0) {
                    if (cta == 0) mbar_arrive_expect_tx(v_full, 2u * (uint32_t)(vb * kHalfBytes));
                    const uint32_t bar = mapa_shared(smem_u32(v_full), 0);
                    for (int j = 0; j < vb; ++j) tma2_2d(vs + j * kHalfBytes, &tv, j * kWideK, row, bar);
                }
                // blocks of b, two to a stage
                int j = 0;
                while (a != kNoMore && ok) {
                    const int a0 = a, j0 = j;
                    if (++j == bb) j = 0, a = ta.next();
                    const int a1 = a, j1 = j;
                    if (a != kNoMore && ++j == bb) j = 0, a = ta.next();
                    turn(a1 != kNoMore ? 2 * kHalfBytes : kHalfBytes);
                    if (ok && lane == 0) {
                        unsigned char* st = sm + st_i * kStageBytes;
                        const uint32_t bar = mapa_shared(smem_u32(full + st_i), 0);
                        tma2_3d(st, &tb, j0 * kWideK, wrow, a0, bar);
                        if (a1 != kNoMore) tma2_3d(st + kHalfBytes, &tb, j1 * kWideK, wrow, a1, bar);
                    }
                    next_stage();
                }
            }
        }
    } else if (warp == 1) {
        if (cta == 0) {
            uint32_t use = 0, n_v = 0;
            for (int64_t tile = tile0; tile < P.n_tiles && ok; tile += tstep, ++use) {
                const uint32_t buf = use & 1u;
                const Tile T = wide_tile(P, tile);
                constexpr uint32_t idesc = idesc_bf16(256, 256);
                TileAdapters ta;
                if (MODE == kLora && tile != tile0) ta.load(P, T.tt, lane);
                ok = __all_sync(0xffffffffu, mbar_wait(acc_empty + buf, ((use >> 1) & 1u) ^ 1u));
                if (!ok) break;
                tc::fence_after();
                const uint32_t d = tm + buf * 256;
                for (int kb = T.kb0; kb < T.kb1; ++kb, next_stage()) {
                    ok = __all_sync(0xffffffffu, mbar_wait(full + st_i, st_ph));
                    if (!ok) break;
                    tc::fence_after();
                    if (lane == 0) {
                        const uint32_t a0 = tc::smem_addr(sm + st_i * kStageBytes), b0 = a0 + kHalfBytes;
#pragma unroll
                        for (int k16 = 0; k16 < kWideK / 16; ++k16)
                            mma2_bf16(d, tc::sdesc(a0 + k16 * 32), tc::sdesc(b0 + k16 * 32), idesc,
                                      kb > T.kb0 || k16 > 0 ? 1u : 0u);
                        commit2(empty + st_i);
                    }
                    __syncwarp();
                }
                if (MODE == kLora && tile == tile0) {
                    griddep_wait();
                    ta.load(P, T.tt, lane);
                }
                if (!ok) break;
                int a = MODE == kLora && T.last ? ta.next() : kNoMore;
                if (a != kNoMore) {
                    ok = __all_sync(0xffffffffu, mbar_wait(v_full, n_v & 1u));
                    ++n_v;
                    if (!ok) break;
                    const uint32_t v0 = tc::smem_addr(vs);
                    // one block of an adapter's b, hi and lo of v against it
                    auto block = [&](int e, int j, uint32_t b0) {
                        uint32_t off[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) off[i] = ~__ballot_sync(0xffffffffu, ta.a[i] == e);
                        if (lane != 0) return;
                        const int steps = min(4, rp - 4 * j);
                        const uint32_t hi = v0 + j * kHalfBytes, lo = vb == 1 ? v0 + rp * 32 : v0 + (bb + j) * kHalfBytes;
                        for (int k16 = 0; k16 < steps; ++k16) {
                            mma2_bf16_lanes(d, tc::sdesc(hi + k16 * 32), tc::sdesc(b0 + k16 * 32), idesc, off);
                            mma2_bf16_lanes(d, tc::sdesc(lo + k16 * 32), tc::sdesc(b0 + k16 * 32), idesc, off);
                        }
                    };
                    int j = 0;
                    while (a != kNoMore) {
                        const int a0 = a, j0 = j;
                        if (++j == bb) j = 0, a = ta.next();
                        const int a1 = a, j1 = j;
                        if (a != kNoMore && ++j == bb) j = 0, a = ta.next();
                        ok = __all_sync(0xffffffffu, mbar_wait(full + st_i, st_ph));
                        if (!ok) break;
                        tc::fence_after();
                        const uint32_t b0 = tc::smem_addr(sm + st_i * kStageBytes);
                        block(a0, j0, b0);
                        if (a1 != kNoMore) block(a1, j1, b0 + kHalfBytes);
                        if (lane == 0) commit2(empty + st_i);
                        __syncwarp();
                        next_stage();
                    }
                    if (!ok) break;
                    if (lane == 0) commit2(v_empty);
                }
                if (lane == 0) commit2(acc_full + buf);
                __syncwarp();
            }
        }
    } else {
        if (kEarly) {
            griddep_wait();
            griddep_launch_dependents();
        }
        const int q4 = warp & 3;  // TMEM lanes 32 q4 .. are this warp's
        unsigned char* store = sm + kStoreOff + q4 * 2 * kStoreBytes;
        const uint32_t empty_bar[2] = {mapa_shared(smem_u32(acc_empty), 0), mapa_shared(smem_u32(acc_empty + 1), 0)};
        uint32_t use = 0, n_store = 0;
        for (int64_t tile = tile0; tile < P.n_tiles; tile += tstep, ++use) {
            const uint32_t buf = use & 1u;
            const Tile T = wide_tile(P, tile);
            constexpr int cols = MODE == kGated ? 128 : 256;  // output columns of the tile
            ok = __all_sync(0xffffffffu, mbar_wait(acc_full + buf, (use >> 1) & 1u));
            if (!ok) break;
            tc::fence_after();
            const int t0 = T.tt * kWideTok + 128 * cta + 32 * q4, n0 = T.wn * cols;
            const uint32_t acc = tc::taddr(tm, 32 * q4, (int)(buf * 256));
            const bool there = t0 + lane < P.n_tok;
            const float4* parts = nullptr;  // of this token, 128 float4 from a group of columns to the next
            if (MODE != kGated && T.at >= 0) {
                // a part of a split tile: into the workspace, and on if it is not the last to arrive
                float4* to = reinterpret_cast<float4*>(P.part) + ((int64_t)T.at * P.split * 2 + cta) * (kPartFloats / 4) +
                             32 * q4 + lane;
                parts = to;
                to += (int64_t)T.part * 2 * (kPartFloats / 4);
                for (int c0 = 0; c0 < 256 && n0 + c0 < P.n_out; c0 += 32) {
                    float v[32];
                    tc::ld32(acc + c0, v);
                    if (there)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            to[(c0 / 4 + i) * 128] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
                tc::fence_before();
                __threadfence();
                __syncwarp();
                int n = 0;
                if (lane == 0) {
                    arrive_cluster(empty_bar[buf]);
                    n = atomicAdd(P.arrived + (T.at * 2 + cta) * 4 + q4, 1);
                }
                n = __shfl_sync(0xffffffffu, n, 0);
                if (n != P.split - 1) continue;
                __threadfence();
            }
            // 32 columns of the accumulator, or the sum of the parts in their order, whoever came last
            auto columns = [&](int c, float v[32]) {
                if (T.at < 0) {
                    tc::ld32(acc + c, v);
                    return;
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.f;
                const int n_parts = there && n0 + c < P.n_out ? P.split : 0;
                for (int p0 = 0; p0 < n_parts; p0 += 4) {  // four parts' loads under way together
                    float4 w[4][8];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (p0 + q < n_parts)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                w[q][i] = __ldcg(parts + (int64_t)(p0 + q) * 2 * (kPartFloats / 4) + (c / 4 + i) * 128);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (p0 + q < n_parts)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                v[4 * i] += w[q][i].x, v[4 * i + 1] += w[q][i].y, v[4 * i + 2] += w[q][i].z, v[4 * i + 3] += w[q][i].w;
                }
            };
            for (int c0 = 0; c0 < cols; c0 += 64) {
                unsigned char* dst = store + (n_store & 1u) * kStoreBytes + lane * 128;
                // the store before the last has read this buffer
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[32];
                    if (MODE == kGated) {
                        uint32_t g[32], u[32];
                        tc::ld32_nowait(acc + c0 + 32 * h, g);
                        tc::ld32_nowait(acc + c0 + 32 * h + 128, u);
                        tc::ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = silu_gate(__uint_as_float(g[i])) * __uint_as_float(u[i]);
                    } else {
                        columns(c0 + 32 * h, v);
                    }
                    if (c0 + 64 >= cols && h == 1 && T.at < 0) {  // the accumulator has been read
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_cluster(empty_bar[buf]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4*>(dst + (((4 * h + i) ^ (lane & 7)) << 4)) = pack8(v + 8 * i);
                }
                // columns past the last whole 16 bytes (a TMA store writes those 16 bytes in full)
                if (n0 + c0 + 64 > P.n_full && there)
                    for (int n = max(P.n_full, n0 + c0); n < min(P.n_out, n0 + c0 + 64); ++n) {
                        const int c = n - n0 - c0;
                        P.out[(int64_t)(t0 + lane) * P.ld + n] =
                            reinterpret_cast<const __nv_bfloat16*>(dst + (((c >> 3) ^ (lane & 7)) << 4))[c & 7];
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (n0 + c0 < P.n_full && t0 < P.n_tok) tma_store_2d(&tout, n0 + c0, t0, dst);
                    bulk_commit();
                }
                ++n_store;
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    tc::fence_before();
    const int bad = __syncthreads_or(!ok);
    if (bad && tid == 0) report_device_status(kDevWaitTimeout);
    cluster_arrive_release();  // no CTA leaves while the other's MMAs or arrivals may still reach it
    cluster_wait_acquire();
    if (warp == 1) dealloc2(tm, 512);
}

// pairs of SMs that can be busy at the same time (the dies' SMs do not all pair up), once per device
template <int MODE>
int pair_count() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    int n = known[dev & 63].load(std::memory_order_acquire);
    if (n > 0) return n;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (sm_count() / 2 > 0 ? sm_count() / 2 : 1));
    cfg.blockDim = dim3(kWideThreads);
    cfg.dynamicSmemBytes = kWideSmem;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, k_wide<MODE>, &cfg) != cudaSuccess || n < 1) n = 1;
    known[dev & 63].store(n, std::memory_order_release);
    return n;
}

template <int MODE>
cudaError_t launch_wide_mode(const WideJob& job, cudaStream_t st) {
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = raise_smem_limit(k_wide<MODE>, kWideSmem, smem_set);
    if (e != cudaSuccess) return e;
    const int pairs = pair_count<MODE>();
    WideArgs P = {};
    P.n_tok = job.n_tok;
    P.n_out = job.n_out;
    P.kb = (job.k + kWideK - 1) / kWideK;
    P.tiles_t = (int32_t)((job.n_tok + kWideTok - 1) / kWideTok);
    P.n_full = job.n_out / 8 * 8;
    P.out = static_cast<__nv_bfloat16*>(job.out);
    P.ld = job.ld;
    P.tok_adapter = job.tok_adapter;
    P.rank = job.rank;
    P.n_adapters = job.n_adapters;
    const WidePlan& plan = job.plan;
    constexpr int cols = MODE == kGated ? 128 : 256;
    P.tiles_n = (job.n_out + cols - 1) / cols;
    P.n_whole = plan.whole;
    P.split = plan.split;
    P.n_tiles = plan.whole + plan.rest * plan.split;
    if (plan.split > 1) {
        P.arrived = static_cast<int32_t*>(job.split_ws);
        P.part = reinterpret_cast<float*>(static_cast<unsigned char*>(job.split_ws) + plan.counter_bytes);
    }
    P.zero = job.zero;
    P.n_zero = job.n_zero;
    P.token_fast = job.n_tok < (MODE == kGated ? 2 : 1) * (int64_t)job.n_out;  // the tokens are the smaller operand
    CUtensorMap mx, mw, mw2, mo, mv, mb;
    bool good = map_rows(&mx, job.x, job.n_tok, job.k, 128) && map_rows(&mw, job.w, job.n_out, job.k, 128) &&
                map_rows(&mo, job.out, job.n_tok, std::max(P.n_full, 8), 32, job.ld);
    if (MODE == kGated) good = good && map_rows(&mw2, job.w2, job.n_out, job.k, 128);
    else mw2 = mw;
    if (MODE == kLora)
        good = good && map_rows(&mv, job.v, job.n_tok, low_row(job.rank), 128) &&
               map_stack(&mb, job.b, job.n_adapters, job.n_out, job.rank, 128);
    else mv = mb = mx;
    if (!good) return cudaErrorInvalidValue;
    const int64_t grid = 2 * std::min<int64_t>(P.n_tiles, pairs);
    return launch_pdl(k_wide<MODE>, dim3((unsigned)grid), dim3(kWideThreads), kWideSmem, st, mx, mw, mw2, mo, mv, mb, P);
}

}  // namespace

constexpr int64_t kPairs = 76;

// Depends on the sizes only, so that a workspace can be sized without a device: 76 pairs, of which a device with others
// makes the same jobs.  Cycles, from measurements of 1 to 1500 tokens: a K block takes 585, and no fewer with fewer columns
// (the tensor cores read the 128 rows of x in the same time for 64 columns as for 256: halves and quarters of tiles in the
// last wave cost as much as whole ones); a job's start and end 2100; parts of a tile, written and read again, 4000 and 4200
// each; an adapter's blocks 128 an MMA and 500 around them; a launch 6 us.  Came to 0.7 to 1.1 of the measured time without adapters, 0.5
// to 1.35 with them (0.5 where every token brings its own, which goes to the other kernel by far).
WidePlan wide_plan(int64_t n_tok, int32_t n_out, int32_t k, bool gated, int32_t rank, int64_t adapters) {
    constexpr int64_t kKBlock = 585, kJob = 2100;
    const int kb = (k + kWideK - 1) / kWideK, cols = gated ? 128 : 256;
    const int64_t tiles = (n_out + cols - 1) / cols * ((n_tok + kWideTok - 1) / kWideTok);
    const int64_t extra = rank > 0 ? adapters * ((rank + 15) / 16 * 256 + 500) : 0;
    WidePlan plan;
    plan.whole = tiles / kPairs * kPairs;
    plan.rest = tiles - plan.whole;
    plan.split = 1;
    int64_t least = -1;
    for (int c = 1; c <= (gated ? 1 : 8) && c <= std::max(1, kb / 2); ++c) {
        const int64_t waves = (plan.rest * c + kPairs - 1) / kPairs;
        const int64_t cost = waves * ((kb + c - 1) / c * kKBlock + kJob) + (waves > 0 ? extra : 0) + (c > 1 ? 4000 + 4200 * c : 0);
        if (least < 0 || cost < least) {
            least = cost;
            plan.split = c;
        }
    }
    plan.counters = plan.split > 1 ? (int32_t)plan.rest * 8 : 0;
    plan.counter_bytes = ((size_t)plan.counters * 4 + 255) & ~(size_t)255;
    plan.ws_bytes = plan.split > 1 ? plan.counter_bytes + (size_t)plan.rest * plan.split * 2 * kPartFloats * 4 : 0;
    plan.us100 = 600 + (plan.whole / kPairs * (kb * kKBlock + kJob + extra) + least) / 19;
    return plan;
}

// The tiles that are left over repeat after kPairs more blocks of 256 tokens at the latest, and adapters cost every split the
// same, so these plans are all there are.
size_t wide_ws_most(int64_t n_tok, int32_t n_out, int32_t k) {
    size_t most = 0;
    for (int64_t t = std::min<int64_t>((n_tok + kWideTok - 1) / kWideTok, kPairs); t > 0; --t)
        most = std::max(most, wide_plan(t * kWideTok, n_out, k, false, 0, 0).ws_bytes);
    return most;
}

cudaError_t take_device_status_wide(unsigned* out) { return take_device_status_tu(out); }

cudaError_t launch_wide(const WideJob& job, cudaStream_t st) {
    if (job.n_tok == 0 || job.n_out == 0) return cudaSuccess;
    return job.rank > 0 ? launch_wide_mode<kLora>(job, st)
                        : job.w2 ? launch_wide_mode<kGated>(job, st) : launch_wide_mode<kPlain>(job, st);
}

}  // namespace gdn
