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
// lora: after the K blocks of x and w come, for each adapter that the tile's tokens use, those of the low-rank
// activations v and of the adapter's b.  The MMA leaves the lanes of all other tokens as they are (its lane mask), so
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
constexpr int kWideStages = 6;
constexpr int kHalfBytes = 128 * kWideK * 2;        // 128 rows of x, or (at most) of the weights
constexpr int kStageBytes = 2 * kHalfBytes;
constexpr int kStoreBytes = 32 * 128;               // 32 tokens x 64 columns
constexpr int kStoreOff = kWideStages * kStageBytes;  // per epilogue warp two of them
constexpr int kBarOff = kStoreOff + 8 * kStoreBytes;  // full[S], empty[S], acc_full[2], acc_empty[2], TMEM address
constexpr int kWideSmem = kBarOff + (2 * kWideStages + 4) * 8 + 16 + 1024;
static_assert(kWideSmem <= 227 * 1024, "shared memory of a CTA");

struct WideArgs {
    int64_t n_tok, n_tiles;
    int32_t n_out;
    int32_t kb;          // 64-wide K blocks
    // Tiles from n_whole on, which would leave pairs idle in a last wave of their own, are cut into `cut` parts of 256 / cut
    // columns each: tile n_whole + i is part i % cut of whole tile n_whole + i / cut.
    int64_t n_whole;
    int32_t cut;
    int32_t tiles_n, tiles_t;
    int32_t token_fast;  // tile order: token blocks fastest (1) or weight blocks fastest (0)
    int32_t n_full;      // columns that go by TMA: n_out rounded down to 16 bytes
    __nv_bfloat16* out;  // the others
    int64_t ld;
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

// What a tile covers.  The smaller operand goes fastest, it is the one that every sweep reads again.
struct Tile {
    int tt;       // token block
    int half;     // weight rows of one CTA: half the accumulator's columns
    int wrow;     // gated: first row of both matrices; else first weight row of the first CTA
    bool narrow;  // cut: another box of weight rows
};
__device__ __forceinline__ Tile wide_tile(const WideArgs& P, int64_t tile, bool gated) {
    int part = 0, cut = 1;
    const bool narrow = tile >= P.n_whole && P.cut > 1;
    if (narrow) {
        cut = P.cut;
        part = (int)((tile - P.n_whole) % cut);
        tile = P.n_whole + (tile - P.n_whole) / cut;
    }
    int wn, tt;
    if (P.token_fast) {
        wn = (int)(tile / P.tiles_t);
        tt = (int)(tile % P.tiles_t);
    } else {
        wn = (int)(tile % P.tiles_n);
        tt = (int)(tile / P.tiles_n);
    }
    const int half = 128 / cut;
    return Tile{tt, half, gated ? wn * 128 + part * half : wn * 256 + part * 2 * half, narrow};
}

// The adapters that a tile's 256 tokens use, by a whole warp: lane l holds those of tokens l, l + 32, ...
struct TileAdapters {
    int a[8], last;
    __device__ __forceinline__ void load(const WideArgs& P, int tt, int lane) {
        last = -1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t t = (int64_t)tt * kWideTok + 32 * j + lane;
            const int v = t < P.n_tok ? P.tok_adapter[t] : -1, e = v & ~kLongRequest;
            a[j] = v >= 0 && e < P.n_adapters ? e : -1;
        }
    }
    // the next one in ascending order (INT_MAX: no more)
    __device__ __forceinline__ int next() {
        int m = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (a[j] > last) m = min(m, a[j]);
        last = __reduce_min_sync(0xffffffffu, m);
        return last;
    }
};

// 8 fp32 -> 16 bytes of bf16
__device__ __forceinline__ uint4 pack8(const float v[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
    k_wide(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw,
           const __grid_constant__ CUtensorMap tw2, const __grid_constant__ CUtensorMap twn,
           const __grid_constant__ CUtensorMap tw2n, const __grid_constant__ CUtensorMap tout,
           const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tb,
           const __grid_constant__ CUtensorMap tbn, const __grid_constant__ WideArgs P) {
    constexpr int S = kWideStages;
    griddep_wait();  // launched with programmatic serialization: nothing is held while kernels ahead still run
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + kBarOff);
    uint64_t* empty = full + S;
    uint64_t* acc_full = empty + S;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(acc_empty + 2);
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
        fence_mbar_init();
    }
    if (warp == 1) alloc2(tslot, 512);
    tc::fence_before();
    __syncthreads();
    cluster_arrive_release();  // the other CTA's barriers and TMEM are ready
    cluster_wait_acquire();
    tc::fence_after();
    griddep_launch_dependents();
    const uint32_t tm = *tslot;
    bool ok = true;

    // blocks of v and b for an adapter: up to 32 ranks as one 64-wide block [hi | lo], else blocks of hi, then of lo
    const int rp = (P.rank + 15) / 16, nb = P.rank <= 32 ? 1 : 2 * ((P.rank + 63) / 64);

    if (warp == 0) {
        uint32_t it = 0;
        // waits for the stage's turn; the first CTA's barrier expects both CTAs' bytes
        auto turn = [&](int s, int half) {
            const bool w = mbar_wait(empty + s, ((it / S) & 1u) ^ 1u);
            ok = __all_sync(0xffffffffu, w);
            if (ok && cta == 0 && lane == 0)
                mbar_arrive_expect_tx(full + s, 2u * (uint32_t)(kHalfBytes + half * kWideK * 2));
        };
        for (int64_t tile = tile0; tile < P.n_tiles && ok; tile += tstep) {
            const Tile T = wide_tile(P, tile, MODE == kGated);
            const int row = T.tt * kWideTok + 128 * cta, wrow = MODE == kGated ? T.wrow : T.wrow + T.half * cta;
            const void* wmap = MODE == kGated && cta == 1 ? (T.narrow ? &tw2n : &tw2) : T.narrow ? &twn : &tw;
            for (int kb = 0; kb < P.kb && ok; ++kb, ++it) {
                const int s = (int)(it % S);
                turn(s, T.half);
                if (ok && lane == 0) {
                    unsigned char* st = sm + s * kStageBytes;
                    const uint32_t bar = mapa_shared(smem_u32(full + s), 0);
                    tma2_2d(st, &tx, kb * kWideK, row, bar);
                    tma2_2d(st + kHalfBytes, wmap, kb * kWideK, wrow, bar);
                }
            }
            if (MODE == kLora && ok) {
                TileAdapters ta;
                ta.load(P, T.tt, lane);
                for (int a = ta.next(); a != 0x7fffffff && ok; a = ta.next())
                    for (int j = 0; j < nb && ok; ++j, ++it) {
                        const int s = (int)(it % S);
                        turn(s, T.half);
                        if (ok && lane == 0) {
                            unsigned char* st = sm + s * kStageBytes;
                            const uint32_t bar = mapa_shared(smem_u32(full + s), 0);
                            tma2_2d(st, &tv, j * kWideK, row, bar);
                            tma2_3d(st + kHalfBytes, T.narrow ? &tbn : &tb, (nb > 1 ? j % (nb / 2) : 0) * kWideK, wrow, a, bar);
                        }
                    }
            }
        }
    } else if (warp == 1) {
        if (cta == 0) {
            uint32_t it = 0, use = 0;
            for (int64_t tile = tile0; tile < P.n_tiles && ok; tile += tstep, ++use) {
                const uint32_t buf = use & 1u;
                const Tile T = wide_tile(P, tile, MODE == kGated);
                const uint32_t idesc = idesc_bf16(256, 2 * T.half);
                ok = __all_sync(0xffffffffu, mbar_wait(acc_empty + buf, ((use >> 1) & 1u) ^ 1u));
                if (!ok) break;
                tc::fence_after();
                const uint32_t d = tm + buf * 256;
                for (int kb = 0; kb < P.kb; ++kb, ++it) {
                    const int s = (int)(it % S);
                    ok = __all_sync(0xffffffffu, mbar_wait(full + s, (it / S) & 1u));
                    if (!ok) break;
                    tc::fence_after();
                    if (lane == 0) {
                        const uint32_t a0 = tc::smem_addr(sm + s * kStageBytes), b0 = a0 + kHalfBytes;
#pragma unroll
                        for (int k16 = 0; k16 < kWideK / 16; ++k16)
                            mma2_bf16(d, tc::sdesc(a0 + k16 * 32), tc::sdesc(b0 + k16 * 32), idesc,
                                      kb > 0 || k16 > 0 ? 1u : 0u);
                        commit2(empty + s);
                    }
                    __syncwarp();
                }
                if (MODE == kLora && ok) {
                    TileAdapters ta;
                    ta.load(P, T.tt, lane);
                    for (int a = ta.next(); a != 0x7fffffff && ok; a = ta.next()) {
                        uint32_t off[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) off[j] = ~__ballot_sync(0xffffffffu, ta.a[j] == a);
                        for (int j = 0; j < nb; ++j, ++it) {
                            const int s = (int)(it % S);
                            ok = __all_sync(0xffffffffu, mbar_wait(full + s, (it / S) & 1u));
                            if (!ok) break;
                            tc::fence_after();
                            if (lane == 0) {
                                const uint32_t a0 = tc::smem_addr(sm + s * kStageBytes), b0 = a0 + kHalfBytes;
                                const int steps = nb == 1 ? rp : min(4, rp - 4 * (j % (nb / 2)));
                                for (int k16 = 0; k16 < steps; ++k16)
                                    mma2_bf16_lanes(d, tc::sdesc(a0 + k16 * 32), tc::sdesc(b0 + k16 * 32), idesc, off);
                                if (nb == 1)
                                    for (int k16 = 0; k16 < steps; ++k16)
                                        mma2_bf16_lanes(d, tc::sdesc(a0 + (rp + k16) * 32), tc::sdesc(b0 + k16 * 32), idesc,
                                                        off);
                                commit2(empty + s);
                            }
                            __syncwarp();
                        }
                    }
                }
                if (!ok) break;
                if (lane == 0) commit2(acc_full + buf);
                __syncwarp();
            }
        }
    } else {
        const int q4 = warp & 3;  // TMEM lanes 32 q4 .. are this warp's
        unsigned char* store = sm + kStoreOff + q4 * 2 * kStoreBytes;
        const uint32_t empty_bar[2] = {mapa_shared(smem_u32(acc_empty), 0), mapa_shared(smem_u32(acc_empty + 1), 0)};
        uint32_t use = 0, n_store = 0;
        for (int64_t tile = tile0; tile < P.n_tiles; tile += tstep, ++use) {
            const uint32_t buf = use & 1u;
            const Tile T = wide_tile(P, tile, MODE == kGated);
            const int half = T.half, cols = MODE == kGated ? half : 2 * half;  // output columns of the tile
            ok = __all_sync(0xffffffffu, mbar_wait(acc_full + buf, (use >> 1) & 1u));
            if (!ok) break;
            tc::fence_after();
            const int t0 = T.tt * kWideTok + 128 * cta + 32 * q4, n0 = T.wrow;
            for (int c0 = 0; c0 < cols; c0 += 64) {
                unsigned char* dst = store + (n_store & 1u) * kStoreBytes + lane * 128;
                // the store before the last has read this buffer
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[32];
                    const uint32_t col = tc::taddr(tm, 32 * q4, (int)(buf * 256) + c0 + 32 * h);
                    if (MODE == kGated) {
                        uint32_t g[32], u[32];
                        tc::ld32_nowait(col, g);
                        tc::ld32_nowait(col + half, u);
                        tc::ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = siluf_(__uint_as_float(g[i])) * __uint_as_float(u[i]);
                    } else {
                        tc::ld32(col, v);
                    }
                    if (c0 + 64 >= cols && h == 1) {  // the accumulator has been read
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_cluster(empty_bar[buf]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4*>(dst + (((4 * h + i) ^ (lane & 7)) << 4)) = pack8(v + 8 * i);
                }
                // columns past the last whole 16 bytes (a TMA store writes those 16 bytes in full)
                if (n0 + c0 + 64 > P.n_full && t0 + lane < P.n_tok)
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

// ---- v = scale A x of the long requests ---------------------------------------------------------------
// A cluster per 128 tokens (TMEM lanes), the rank being the MMA's N side; as above, an adapter's MMAs leave the lanes of
// other tokens alone.  The product is small and its tokens are read once per adapter of a tile, so it is bound by how many
// loads are in flight: K is split over the cluster until the GPU is full, and the fp32 parts are joined through
// distributed shared memory in the order of the ranks, each CTA finishing its share of the tokens.
constexpr int kLowStages = 4;
constexpr int kLowStage = 2 * kHalfBytes;
constexpr int kLowBar = kLowStages * kLowStage;  // full[S], empty[S], done, TMEM address
constexpr int kLowSmem = kLowBar + (2 * kLowStages + 1) * 8 + 8 + 1024;
static_assert(128 * 128 * 4 <= kLowBar, "a partial block over the ring");

struct WideLowArgs {
    int64_t n_tok;
    const int32_t* tok_adapter;
    const float* scale;
    __nv_bfloat16* v;
    int32_t kb, rank, ks, n_adapters;
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

__global__ void __launch_bounds__(kWideThreads, 1)
    k_wide_low(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap ta,
               const __grid_constant__ WideLowArgs P) {
    constexpr int S = kLowStages;
    constexpr uint32_t COLS = 128;
    griddep_wait();
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + kLowBar);
    uint64_t* empty = full + S;
    uint64_t* done = empty + S;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rp = (P.rank + 15) / 16 * 16, ks = P.ks, rank = (int)(blockIdx.x % ks);
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
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    griddep_launch_dependents();
    const uint32_t tm = *tslot;
    bool ok = true;

    // the adapters of the tile's long requests: lane l holds those of tokens l, l + 32, ...
    auto adapter_of = [&](int64_t t) {
        const int v = t < P.n_tok ? P.tok_adapter[t] : -1, e = v & ~kLongRequest;
        return v >= 0 && (v & kLongRequest) && e < P.n_adapters ? e : -1;
    };
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
                    unsigned char* st = sm + s * kLowStage;
                    mbar_arrive_expect_tx(full + s, (uint32_t)(kHalfBytes + rp * kWideK * 2));
                    tma_tile_2d(st, &tx, kb * kWideK, (int)t0, full + s);
                    tma_tile_3d(st + kHalfBytes, &ta, kb * kWideK, 0, e, full + s);
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
                    const uint32_t a0 = tc::smem_addr(sm + s * kLowStage), b0 = a0 + kHalfBytes;
#pragma unroll
                    for (int k16 = 0; k16 < kWideK / 16; ++k16)
                        mma_bf16_lanes(tm, tc::sdesc(a0 + k16 * 32), tc::sdesc(b0 + k16 * 32), idesc,
                                       kb > kb0 || k16 > 0 ? 1u : 0u, off);
                    tc::commit(empty + s);
                }
                __syncwarp();
            }
        }
        if (ok && lane == 0) tc::commit(done);
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
        const int lo = P.rank <= 32 ? rp : (P.rank + 63) / 64 * 64, row = low_row(P.rank), mine = 128 / ks;
        const uint32_t own = smem_u32(sm);
        for (int i = tid; i < mine * (rp / 8); i += kWideThreads) {
            const int c0 = i / mine * 8, tok = rank * mine + i % mine, e = adapter_of(t0 + tok);
            if (e < 0) continue;
            float v[8] = {}, l[8];
            for (int r = 0; r < ks; ++r) {
                const uint32_t src = (ks > 1 ? mapa_shared(own, r) : own) + (uint32_t)(c0 * 128 + tok) * 4;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float p;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p) : "r"(src + j * 512) : "memory");
                    v[j] += p;
                }
            }
            const float scale = P.scale ? P.scale[e] : 1.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] *= scale;
                const float h = __bfloat162float(__float2bfloat16_rn(v[j]));
                l[j] = isfinite(h) ? v[j] - h : 0.f;
            }
            __nv_bfloat16* dst = P.v + (t0 + tok) * row + c0;
            *reinterpret_cast<uint4*>(dst) = pack8(v);
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

// bf16 [n][rows][cols], boxes of 64 columns x box_rows of one matrix
bool map_stack(CUtensorMap* m, const void* base, int64_t n, int64_t rows, int64_t cols, int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * (cuuint64_t)rows * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
    constexpr int cols = MODE == kGated ? 128 : 256;
    P.tiles_n = (job.n_out + cols - 1) / cols;
    const int64_t tiles = (int64_t)P.tiles_n * P.tiles_t;
    P.n_whole = tiles / pairs * pairs;
    // the rest, cut where its waves then cost less; a tile costs its columns and a start worth about 24
    const int64_t rest = tiles - P.n_whole;
    int64_t least = -1;
    for (int cut = 1; cut <= (MODE == kGated ? 2 : 4); cut *= 2) {  // (results are stored in pieces of 64 columns)
        const int64_t cost = (rest * cut + pairs - 1) / pairs * (256 / cut + 24);
        if (least < 0 || cost < least) {
            least = cost;
            P.cut = cut;
        }
    }
    P.n_tiles = P.n_whole + rest * P.cut;
    P.token_fast = job.n_tok < (MODE == kGated ? 2 : 1) * (int64_t)job.n_out;  // the tokens are the smaller operand
    CUtensorMap mx, mw, mw2, mwn, mw2n, mo, mv, mb, mbn;
    bool good = map_rows(&mx, job.x, job.n_tok, job.k, 128) && map_rows(&mw, job.w, job.n_out, job.k, 128) &&
                map_rows(&mo, job.out, job.n_tok, std::max(P.n_full, 8), 32, job.ld);
    if (MODE == kGated) good = good && map_rows(&mw2, job.w2, job.n_out, job.k, 128);
    else mw2 = mw;
    if (MODE == kLora)
        good = good && map_rows(&mv, job.v, job.n_tok, low_row(job.rank), 128) &&
               map_stack(&mb, job.b, job.n_adapters, job.n_out, job.rank, 128);
    else mv = mb = mx;
    mwn = mw, mw2n = mw2, mbn = mb;
    if (P.cut > 1) {
        const int box = 128 / P.cut;
        good = good && map_rows(&mwn, job.w, job.n_out, job.k, box);
        if (MODE == kGated) good = good && map_rows(&mw2n, job.w2, job.n_out, job.k, box);
        if (MODE == kLora) good = good && map_stack(&mbn, job.b, job.n_adapters, job.n_out, job.rank, box);
    }
    if (!good) return cudaErrorInvalidValue;
    const int64_t grid = 2 * std::min<int64_t>(P.n_tiles, pairs);
    return launch_pdl(k_wide<MODE>, dim3((unsigned)grid), dim3(kWideThreads), kWideSmem, st, mx, mw, mw2, mwn, mw2n, mo, mv,
                      mb, mbn, P);
}

}  // namespace

cudaError_t take_device_status_wide(unsigned* out) { return take_device_status_tu(out); }

cudaError_t launch_wide(const WideJob& job, cudaStream_t st) {
    if (job.n_tok == 0 || job.n_out == 0) return cudaSuccess;
    return job.rank > 0 ? launch_wide_mode<kLora>(job, st)
                        : job.w2 ? launch_wide_mode<kGated>(job, st) : launch_wide_mode<kPlain>(job, st);
}

cudaError_t launch_wide_low(const LowJob& job, cudaStream_t st) {
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t e = raise_smem_limit(k_wide_low, kLowSmem, smem_set);
    if (e != cudaSuccess) return e;
    CUtensorMap mx, ma;
    if (!map_rows(&mx, job.x, job.n_tok, job.k, 128) ||
        !map_stack(&ma, job.a, job.n_adapters, job.rank, job.k, (job.rank + 15) / 16 * 16))
        return cudaErrorInvalidValue;
    WideLowArgs P = {};
    P.n_tok = job.n_tok;
    P.tok_adapter = job.tok_adapter;
    P.scale = job.scale;
    P.v = static_cast<__nv_bfloat16*>(job.v);
    P.kb = (job.k + kWideK - 1) / kWideK;
    P.rank = job.rank;
    P.n_adapters = job.n_adapters;
    const int64_t tiles = (job.n_tok + 127) / 128;
    P.ks = 1;
    while (P.ks < 8 && tiles * P.ks * 2 <= sm_count() && P.kb >= P.ks * 4) P.ks *= 2;
    return launch_pdl_cluster(k_wide_low, dim3((unsigned)(tiles * P.ks)), dim3(kWideThreads), kLowSmem, P.ks, st, mx, ma, P);
}

}  // namespace gdn
