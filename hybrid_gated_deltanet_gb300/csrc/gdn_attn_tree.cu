// gdn_attn_tree.cu -- attention of a tree of drafted tokens per sequence over its paged KV cache:
// node i attends to the cached tokens 0 .. ctx - 1, to its ancestors and to itself
// ("Forge: how I wrote my own inference engine and overtook llama.cpp", 27 August: a draft is
// verified as a chunk of rows over the cache; here the rows form a tree).
//
// The rows of a kv-head are the (node, query head) pairs of its group: up to 64 nodes x G heads, cut
// into tiles of 128, the M of one tcgen05 product.  K and V are read once per row tile, and one row tile
// holds everything up to 128 rows, so that short trees are bound by HBM (M flops per byte against a ridge of
// about 280) and large ones by the tensor cores.
//
// Work: every (sequence, kv-head, row tile) is a list of key tiles (its context's, then one with the nodes
// themselves).  While there is an SM for each list, lists are cut into equal pieces, one per worker (a CTA), as few as
// balance allows; the row tiles of a kv-head are cut at the same places, so their reads of K and V come at the same time
// and meet in L2.  With more lists they are laid end to end and cut into equal runs, whatever the mix of lengths.
// Us, pieces against runs: 16 sequences of up to 8192 tokens, two row tiles of d = 128, 50 against 61; 4 of up to
// 32768, six row tiles of d = 256, 90 against 183; one of 32768, one row tile, 36 against 39.
// A list that lies with one worker is finished by it; one that is cut leaves (maximum, sum, unnormalised O) per part
// in the workspace and k_attn_tree_join joins the parts in order (no atomics: results do not change from call to call).
//
// Measured: 64 nodes over 4 x 32768 tokens (24 / 2 heads of 256) 88 us, 0.90 PFLOP/s: its longest piece has 74 tiles of 64 keys
// (65.7 were equal shares) at 1820 cycles each, 1410 of them products (16 of N = 64 and 4 of N = 256), about 66 us, and the
// rest is the start, the last tile's chain and the join; 24 nodes over 16 x 8192 (32 / 4 heads of 128) 50 us: the longest piece
// has 32 tiles where equal shares had 23.3, each a chain of product, softmax and product (the tensor cores are 22% busy); 16
// nodes over 16 x 8192 (16 / 4 heads of 256) 65 us, 4.7 TB/s, and over 64 x 2048 (runs: 256 lists) 88 us, 3.9 TB/s; a call of one
// list per SM is bound by latency (one tree of 8 nodes over 300 tokens: 12.1 us).
#include <cuda_bf16.h>

#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_tc.cuh"
#include "gdn_tma.cuh"

namespace gdn {
namespace {

constexpr int kTreeCtas = 152;    // one CTA per SM (a constant: the workspace's size is known without a device)
constexpr int kTreeMinTiles = 2;  // fewest key tiles of a worker's run (us, 2 x 1000 tokens: 1 15.4, 2 14.8; an earlier build 4 17.2 against 15.5)
// lists of up to this many tiles are not cut while every list has an SM: nothing to join then (us, whole against cut: 6
// tiles 12.1 against 13.5, 9 tiles 14.0 against 14.2, 17 tiles 20.2 against 14.8)
constexpr int kTreeWhole = 8;

struct AttnTreeArgs {
    const __nv_bfloat16* q;      // [N][Hq][D]
    const __nv_bfloat16* v_new;  // [N][Hkv][D]
    const int32_t* block_table;  // [B][max_pages]
    const int32_t* cu_nodes;
    const int32_t* parents;
    const int32_t* ctx_lens;
    __nv_bfloat16* o;  // [N][Hq][D]
    int4* share;       // [worker][2]: workers of the list that its share begins in, row tile, kv-head; first row, nodes
    float* part;       // [worker][2][D + 2][128]: O by columns, then maximum and sum
    int B, Hq, Hkv, G, W, page, R, max_pages, n_pages, n_nodes, max_nodes, max_ctx;
    int whole;          // > 0: worker w takes list w whole (few short lists: nothing to join), of this many per kv-head
    int even;           // lists in equal pieces (at most W lists); else equal runs of all lists
    float scale_log2;   // scale * log2(e)
};

template <int D>
struct TreeLay {
    static constexpr int NCH = D / 64;             // 64-column chunks of a row (128 bytes)
    static constexpr int BK = D == 256 ? 64 : 128; // keys per tile: 32 KB of K and 32 KB of V either way
    static constexpr int GRP = NCH * 1024;         // 8 key rows: NCH swizzle atoms of 8 x 128 bytes
    static constexpr int TILE = BK / 8 * GRP;
    static constexpr int QATOM = 128 * 128;
    static constexpr int Q = 0;                    // [chunk][128 rows][128 bytes], swizzled
    static constexpr int K = Q + NCH * QATOM;      // 2 stages, [8-row group][chunk][8][128 bytes], swizzled
    static constexpr int V = K + 2 * TILE;         // 2 stages, the same layout
    static constexpr int BAR = V + 2 * TILE;
    static constexpr int MREF = BAR + 40 * 8;      // reference maximum of each row
    static constexpr int LSUM = MREF + 128 * 4;    // sums of the rows, per softmax group
    static constexpr int GONE = LSUM + 256 * 4;    // 4 slots: runs of a tile without keys
    static constexpr int BAD = GONE + 4 * 8;       // 4 slots: nodes with an infinite or NaN value
    static constexpr int ANC = BAD + 4 * 8;        // 4 slots: line of each node (64-bit masks)
    static constexpr int UP = ANC + 4 * 64 * 8;
    static constexpr int SMEM_ALLOC = UP + 64 * 4 + 1024;
    static constexpr int O_COL = 2 * BK;           // TMEM: S of two tiles, O, P of two tiles (2 bf16 to a column)
    static constexpr int P_COL = O_COL + D;
    static constexpr int TMEM_COLS = 512;
    static_assert(P_COL + BK <= TMEM_COLS, "TMEM");
    static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory");
};

// sequence b: rows, context and key tiles (0: skipped)
template <int BK>
__device__ __forceinline__ int tree_tiles(const AttnTreeArgs& A, int b, int& first, int& n, int& ctx) {
    first = A.cu_nodes[b];
    const long long cnt = (long long)A.cu_nodes[b + 1] - first;
    ctx = A.ctx_lens[b];
    if (first < 0 || cnt < 1 || cnt > A.max_nodes || first + cnt > A.n_nodes || ctx < 0 || ctx > A.max_ctx ||
        ctx > (long long)A.max_pages * A.page) {
        n = 0;
        return 0;
    }
    n = (int)cnt;
    return (ctx + BK - 1) / BK + 1;
}

// lists of a sequence: a list per kv-head and row tile
__device__ __forceinline__ int tree_lists(const AttnTreeArgs& A, int n) { return A.Hkv * ((n * A.G + 127) / 128); }

// sum of v over the block's threads, and of the threads before this one
template <int THREADS>
__device__ __forceinline__ void tree_scan(long long v, long long* s_warp, long long& before, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
    }
    __syncthreads();  // s_warp may be in use
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    before = incl - v;
    total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) before += s_warp[i];
        total += s_warp[i];
    }
}

// one piece of a worker's share: tiles t0 .. t1 - 1 of the nt of list (b, kvh), rows 128 rt ..
struct TreeSeg {
    int b, kvh, rt, t0, t1, nt, first, n, ctx;
};

// worker w's share: `left` tiles, of which `seg` is the first piece
struct TreeRun {
    TreeSeg seg;
    long long left;
    int first, last;  // workers that hold the list the share begins in
};

// the piece that begins at tile t0 of list `list` of sequence seg.b (seg.nt, first, n and ctx are known)
__device__ __forceinline__ void tree_piece(const AttnTreeArgs& A, TreeSeg& seg, int list, int t0, long long left) {
    const int per_head = (seg.n * A.G + 127) >> 7;
    seg.kvh = per_head == 1 ? list : list / per_head;
    seg.rt = list - seg.kvh * per_head;
    seg.t0 = t0;
    seg.t1 = (int)min((long long)seg.nt, t0 + left);
}

// ceil(a / per), rcp about 1 / per: exact up to 2^22, and not below 2^22 above that
__device__ __forceinline__ uint32_t tree_div_up(uint32_t a, uint32_t per, float rcp) {
    const uint32_t x = a + per - 1;
    uint32_t q = (uint32_t)((float)x * rcp);
    if ((q + 1) * per <= x) ++q;
    if (q * per > x) --q;
    return q;
}

// A.even: worker w takes piece w.  Every warp works it out by itself (there are at most kTreeCtas sequences, PER to a
// lane): loads of one latency, then a bisection for the shortest pieces of which there are at most W
template <int BK, int PER>
__device__ __forceinline__ TreeRun tree_run_even(const AttnTreeArgs& A, int w) {
    const int lane = threadIdx.x & 31, each = (A.B + 31) / 32;
    uint32_t nt[PER], lists[PER], most = kTreeMinTiles, tiles_here = 0, lists_here = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int b = lane * each + e;
        int first, n = 0, ctx;
        nt[e] = e < each && b < A.B ? tree_tiles<BK>(A, b, first, n, ctx) : 0;
        lists[e] = tree_lists(A, n);
        most = max(most, nt[e]);
        tiles_here += lists[e] * nt[e];  // (at most kTreeCtas lists of 2^24 tiles: 32 bits hold the sum)
        lists_here += lists[e];
    }
    auto count = [&](uint32_t per) {  // pieces of this lane's sequences
        const float rcp = __fdividef(1.f, (float)per);
        uint32_t c = 0;
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (e < each) c += lists[e] * tree_div_up(nt[e], per, rcp);
        return c;
    };
    // at least tiles / W; and tiles / (W - lists) is enough, since rounding up adds less than a piece per list; and so is
    // one piece per list
    const uint32_t tiles_all = __reduce_add_sync(0xffffffffu, tiles_here), lists_all = __reduce_add_sync(0xffffffffu, lists_here);
    uint32_t lo = max((uint32_t)kTreeMinTiles, (tiles_all + A.W - 1) / A.W), hi = __reduce_max_sync(0xffffffffu, most);
    if (lists_all < (uint32_t)A.W) hi = min(hi, tiles_all / (A.W - lists_all) + 1);
    hi = max(hi, lo);
    while (lo < hi) {
        const uint32_t per = (lo + hi) / 2;
        if (__reduce_add_sync(0xffffffffu, count(per)) <= (uint32_t)A.W)
            hi = per;
        else
            lo = per + 1;
    }
    const uint32_t mine = count(lo);
    uint32_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
    }
    const unsigned owner = __ballot_sync(0xffffffffu, (uint32_t)w >= incl - mine && (uint32_t)w < incl);
    TreeRun run;
    run.left = 0;
    if (owner == 0u) return run;
    const float rcp = __fdividef(1.f, (float)lo);
    uint32_t at = incl - mine, piece = 0, pieces = 1, list = 0;
    int b = 0;
    bool found = false;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        if (e >= each) break;
        const uint32_t per_list = tree_div_up(nt[e], lo, rcp), len = lists[e] * per_list;
        if (!found && (uint32_t)w >= at && (uint32_t)w < at + len) {
            found = true;
            b = lane * each + e;
            pieces = per_list;
            list = ((uint32_t)w - at) / per_list;
            piece = (uint32_t)w - at - list * per_list;
        }
        at += len;
    }
    const int src = __ffs(owner) - 1;
    run.seg.b = __shfl_sync(0xffffffffu, b, src);
    pieces = __shfl_sync(0xffffffffu, pieces, src);
    piece = __shfl_sync(0xffffffffu, piece, src);
    list = __shfl_sync(0xffffffffu, list, src);
    run.seg.nt = tree_tiles<BK>(A, run.seg.b, run.seg.first, run.seg.n, run.seg.ctx);
    // (at most 2^24 tiles and kTreeCtas pieces: the products fit)
    const uint32_t tiles = run.seg.nt, t0 = tiles * piece / pieces, t1 = tiles * (piece + 1) / pieces;
    run.left = t1 - t0;
    tree_piece(A, run.seg, (int)list, (int)t0, run.left);
    run.first = w - (int)piece;
    run.last = run.first + (int)pieces - 1;
    return run;
}

// All threads of the block call it.
template <int D, int THREADS>
__device__ __forceinline__ TreeRun tree_run(const AttnTreeArgs& A, int w) {
    constexpr int BK = TreeLay<D>::BK;
    __shared__ long long s_warp[THREADS / 32], s_rem, s_left;
    __shared__ int s_b, s_first, s_last;
    TreeRun run;
    const int tid = threadIdx.x;
    int first, n, ctx;
    if (A.whole) {
        const int lists = A.Hkv * A.whole, b = w / lists, at = w - b * lists;
        run.seg.b = b;
        run.seg.nt = tree_tiles<BK>(A, b, run.seg.first, run.seg.n, run.seg.ctx);
        run.left = at < tree_lists(A, run.seg.n) ? run.seg.nt : 0;
        if (run.left > 0) tree_piece(A, run.seg, at, 0, run.left);
        run.first = run.last = w;
        return run;
    }
    // (run once, the code costs its fetch: the short form is a fifth of the other)
    if (A.even) return A.B <= 32 ? tree_run_even<BK, 1>(A, w) : tree_run_even<BK, (kTreeCtas + 31) / 32>(A, w);
    // each thread sums some sequences; a scan of the threads' sums finds the one that holds the start
    const int each = (A.B + THREADS - 1) / THREADS;
    const int b0 = min(A.B, tid * each), b1 = min(A.B, b0 + each);
    long long sum = 0, before, total;
    for (int b = b0; b < b1; ++b) {
        const int nt = tree_tiles<BK>(A, b, first, n, ctx);
        sum += (long long)nt * tree_lists(A, n);
    }
    tree_scan<THREADS>(sum, s_warp, before, total);
    const long long per = max((long long)kTreeMinTiles, (total + A.W - 1) / A.W), start = w * per;
    if (tid == 0) s_left = 0;
    __syncthreads();
    if (start < total && before <= start && start < before + sum) {
        long long at = before;
        for (int b = b0; b < b1; ++b) {
            const int nt = tree_tiles<BK>(A, b, first, n, ctx);
            const long long len = (long long)nt * tree_lists(A, n);
            if (start < at + len) {
                const long long in = (start - at) % nt;  // tiles of the list that lie before the share
                s_b = b;
                s_rem = start - at;
                s_left = min(per, total - start);
                s_first = (int)((start - in) / per);
                s_last = (int)((start - in + nt - 1) / per);
                break;
            }
            at += len;
        }
    }
    __syncthreads();
    run.left = s_left;
    run.first = s_first;
    run.last = s_last;
    if (run.left > 0) {
        run.seg.b = s_b;
        run.seg.nt = tree_tiles<BK>(A, s_b, run.seg.first, run.seg.n, run.seg.ctx);
        const long long list = s_rem / run.seg.nt;
        tree_piece(A, run.seg, (int)list, (int)(s_rem - list * run.seg.nt), run.left);
    }
    return run;
}

// the pieces of a worker's share, one after another
template <int BK>
struct TreeWalk {
    const AttnTreeArgs& A;
    TreeSeg at;  // the next piece
    long long left;
    __device__ TreeWalk(const AttnTreeArgs& a, const TreeRun& r) : A(a), at(r.seg), left(r.left) {}
    __device__ bool next(TreeSeg& s) {
        if (left <= 0) return false;
        s = at;
        left -= at.t1 - at.t0;
        if (left > 0) {  // on to the next list, or the next sequence that has one
            int list = at.kvh * ((at.n * A.G + 127) >> 7) + at.rt + 1;
            while (list >= tree_lists(A, at.n)) {
                if (++at.b >= A.B) {
                    left = 0;
                    return true;
                }
                at.nt = tree_tiles<BK>(A, at.b, at.first, at.n, at.ctx);
                list = 0;
            }
            tree_piece(A, at, list, 0, left);
        }
        return true;
    }
};

__device__ __forceinline__ uint64_t tree_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3FFF) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;  // 128-byte swizzle
    return d;
}

__device__ __forceinline__ float tree_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tree_tma_5d(void* dst, const CUtensorMap* map, int row8, int line, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, "
        "%4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row8), "r"(line), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tree_tma_4d(void* dst, const CUtensorMap* map, int row, int head, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %2, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(head), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tree_prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// The warp that issues products runs converged and one elected lane issues: 48 cycles an instruction at N = 64,
// the rate of the product itself (67 from a branch on the lane index, 82 with a predicate on each instruction).
__device__ __forceinline__ bool tree_elect() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}
// a product with A in TMEM (lane = row, two bf16 of K to a 32-bit column)
__device__ __forceinline__ void tree_mma_ta(uint32_t d, uint32_t a, uint64_t bd, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(bd), "r"(idesc), "r"(acc)
        : "memory");
}

// 32 consecutive columns of this warp's lanes, no wait
__device__ __forceinline__ void tree_st32(uint32_t ta, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(ta),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// one column of this warp's lanes
__device__ __forceinline__ uint32_t tree_ld1(uint32_t ta) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n tcgen05.wait::ld.sync.aligned;" : "=r"(r) : "r"(ta) : "memory");
    return r;
}

// 16 bytes from global to shared memory, or 16 zeros
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// an infinity or NaN among the two bf16 of a word (all exponent bits set), as a mask of the halves
__device__ __forceinline__ uint32_t nonfinite2(uint32_t u) {
    return ((u & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((u & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// Warp 0 loads K tiles, warp 10 V tiles (and works out the nodes' lines), warps 1 and 11 issue the two products, and
// two groups of four warps (2..5 and 6..9, thread = row) take the tiles in turn, so that one group's softmax runs
// while the other waits, loads or stores.  Tile `it` of the CTA uses group, stage, S and P buffer and barrier it & 1:
//   full_k, full_v   the tile's copies have landed
//   s_done           S = Q K^T is in TMEM (and K's stage is free)
//   s_read           the group has read S for the last time (and S's buffer is free)
//   decided          (per 32 rows) the rows' reference maxima after this tile are in shared memory
//   p_ready          P is in TMEM, O is rescaled, V has no row without a key
//   pv_done          O += P V is done (V's stage and P's buffer are free)
// Every wait is bounded: a role that gives up stops waiting, and the CTA still runs to its end.
constexpr int kTreeThreads = 384;

template <int D>
__global__ void __launch_bounds__(kTreeThreads, 1)
    k_attn_tree(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                const __grid_constant__ CUtensorMap tkn, const __grid_constant__ CUtensorMap tvn,
                const __grid_constant__ AttnTreeArgs A) {
    using Ly = TreeLay<D>;
    constexpr int NCH = Ly::NCH, BK = Ly::BK;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Ly::BAR);
    uint64_t *full_k = bars, *full_v = bars + 2, *s_done = bars + 4, *s_read = bars + 6, *pv_done = bars + 8,
             *p_ready = bars + 10, *anc_ready = bars + 12, *q_ready = bars + 14, *o_free = bars + 15, *gone_ready = bars + 16,
             *decided = bars + 20;  // [group][quarter of the rows]
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 28);
    float* s_mref = reinterpret_cast<float*>(sm + Ly::MREF);
    float* s_l = reinterpret_cast<float*>(sm + Ly::LSUM);
    unsigned* s_gone = reinterpret_cast<unsigned*>(sm + Ly::GONE);
    unsigned long long* s_bad = reinterpret_cast<unsigned long long*>(sm + Ly::BAD);
    unsigned long long* s_anc = reinterpret_cast<unsigned long long*>(sm + Ly::ANC);
    int* s_up = reinterpret_cast<int*>(sm + Ly::UP);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(full_k + i, 1);
            mbar_init(full_v + i, 1);
            mbar_init(s_done + i, 1);
            mbar_init(s_read + i, 4);  // one arrival per warp of the group
            mbar_init(pv_done + i, 1);
            mbar_init(p_ready + i, 4);
            mbar_init(anc_ready + i, 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(gone_ready + i, 1);
        for (int i = 0; i < 8; ++i) mbar_init(decided + i, 1);
        mbar_init(q_ready, 8);
        mbar_init(o_free, 8);
        fence_mbar_init();
    }
    if (tid == 32) {
        tree_prefetch_map(&tk);
        tree_prefetch_map(&tv);
        tree_prefetch_map(&tkn);
        tree_prefetch_map(&tvn);
    }
    __syncthreads();
    griddep_wait();  // launched with programmatic serialization: what is above runs beside the kernel before
    griddep_launch_dependents();
    const TreeRun run = tree_run<D, kTreeThreads>(A, blockIdx.x);
    if (A.share && tid == 352) {  // for the join
        const bool any = run.left > 0;
        A.share[2 * blockIdx.x] = any ? make_int4(run.first, run.last, run.seg.rt, run.seg.kvh) : make_int4(-2, 0, 0, 0);
        A.share[2 * blockIdx.x + 1] = any ? make_int4(run.seg.first, run.seg.n, 0, 0) : make_int4(0, 0, 0, 0);
    }
    if (run.left <= 0) return;  // (the same for all threads)
    uint32_t tm = 0;
    if (warp != 0 && warp != 10) {  // (the warps that load need no TMEM and do not wait for it)
        if (warp == 1) tc::alloc(tslot, Ly::TMEM_COLS);
        tc::fence_before();
        named_bar_sync(2, kTreeThreads - 64);
        tc::fence_after();
        tm = *tslot;
    }
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {  // warp-wide; after a failure nothing waits any more
        if (ok && !__all_sync(0xffffffffu, mbar_test(bar, (uint32_t)(phase & 1))))
            ok = __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)(phase & 1)));
        return ok;
    };

    // key tile j of a segment: lane i looks up the page of its run of R rows; -1: no such run, past the context, or a
    // page outside the pool
    const int nseg = BK / A.R;
    auto lane_page = [&](const TreeSeg& s, int j) -> int {
        const int pos = j * BK + lane * A.R;
        if (lane >= nseg || j >= s.t1 || pos >= s.ctx) return -1;
        const int pid = __ldg(A.block_table + (size_t)s.b * A.max_pages + pos / A.page);
        return (pid >= 0 && pid < A.n_pages) ? pid : -1;
    };
    // keys of tile j, and their steps of 16 in P V (rows past the last step are not read)
    auto keys_of = [&](const TreeSeg& s, int j) { return j == s.nt - 1 ? s.n : min(BK, s.ctx - j * BK); };
    TreeWalk<BK> walk(A, run);
    TreeSeg s;

    if (warp == 0 || warp == 10) {
        // ---- K or V tiles into the two stages -------------------------------------------
        const bool is_k = warp == 0;
        const CUtensorMap* pool_map = is_k ? &tk : &tv;
        const CUtensorMap* new_map = is_k ? &tkn : &tvn;
        unsigned char* ring = sm + (is_k ? Ly::K : Ly::V);
        uint64_t *full = is_k ? full_k : full_v, *freed = is_k ? s_done : pv_done;
        int it = 0, tails = 0;
        while (ok && walk.next(s)) {
            int pid_next = lane_page(s, s.t0);
            for (int j = s.t0; j < s.t1; ++j, ++it) {
                const int pid = pid_next;
                pid_next = lane_page(s, j + 1);
                const int st = it & 1;
                if (it >= 2 && !wait(freed + st, (it - 2) >> 1)) break;
                unsigned char* dst = ring + st * Ly::TILE;
                const unsigned have = __ballot_sync(0xffffffffu, pid >= 0);
                if (is_k && lane == 0) {  // (S of tile it - 2 is done, so tile it - 4 was read and with it this slot)
                    s_gone[it & 3] = ~have;
                    mbar_arrive(gone_ready + (it & 3));
                }
                if (j < s.nt - 1) {
                    if (lane == 0) mbar_arrive_expect_tx(full + st, (uint32_t)(__popc(have) * A.R * D * 2));
                    __syncwarp();
                    if (pid >= 0)
                        tree_tma_5d(dst + lane * (A.R / 8) * Ly::GRP, pool_map, (j * BK + lane * A.R) % A.page / 8,
                                    pid * A.Hkv + s.kvh, full + st);
                    continue;
                }
                const int groups = (s.n + 7) / 8;
                if (lane == 0) mbar_arrive_expect_tx(full + st, (uint32_t)(groups * 8 * D * 2));
                __syncwarp();
                if (lane < groups) tree_tma_4d(dst + lane * Ly::GRP, new_map, s.first + 8 * lane, s.kvh, full + st);
                if (is_k) continue;
                // the line of every node: six rounds of doubling, two nodes to a lane.  Slots are used in turn: the
                // segment that used this one four tails ago was finished before pv_done(it - 2)
                unsigned long long* anc = s_anc + (tails & 3) * 64;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 32 * e + lane;
                    int up = -1;
                    if (i < s.n) {
                        const int p = A.parents[s.first + i];
                        up = p >= 0 && p < i ? p : -1;
                    }
                    s_up[i] = up;
                    anc[i] = i < s.n ? 1ull << i : 0ull;
                }
                if (lane == 0) s_bad[tails & 3] = 0ull;
                __syncwarp();
                for (int step = 0; step < 6; ++step) {
                    unsigned long long m[2];
                    int up[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int i = 32 * e + lane, p = s_up[i];
                        m[e] = anc[i] | (p >= 0 ? anc[p] : 0ull);
                        up[e] = p >= 0 ? s_up[p] : -1;
                    }
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        anc[32 * e + lane] = m[e];
                        s_up[32 * e + lane] = up[e];
                    }
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(anc_ready + (tails & 1));
                ++tails;
            }
        }
        // copies still in flight land before the CTA leaves
        for (int i = max(0, it - 2); i < it; ++i) mbar_wait(full + (i & 1), (uint32_t)((i >> 1) & 1));
    } else if (warp == 1) {
        // ---- S = Q K^T ----------------------------------------------------------------------
        constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BK >> 3) << 17) |
                                   ((uint32_t)(128 >> 4) << 24);
        // descriptors: only the start address (in 16-byte units, the low bits) changes
        const uint64_t dq = tc::sdesc(tc::smem_addr(sm + Ly::Q)), dk = tree_desc(tc::smem_addr(sm + Ly::K), 16, Ly::GRP);
        int it = 0, seg = 0;
        while (ok && walk.next(s)) {
            if (!wait(q_ready, seg)) break;
            ++seg;
            for (int j = s.t0; j < s.t1; ++j, ++it) {
                const int st = it & 1;
                if (!wait(full_k + st, it >> 1) || (it >= 2 && !wait(s_read + st, (it - 2) >> 1))) break;
                tc::fence_after();
                if (tree_elect()) {
                    const uint64_t kb = dk + ((uint32_t)(st * Ly::TILE) >> 4);
#pragma unroll
                    for (int kd = 0; kd < D / 16; ++kd)
                        tc::mma_f16(tm + st * BK, dq + (uint32_t)(((kd >> 2) * Ly::QATOM + (kd & 3) * 32) >> 4),
                                    kb + (uint32_t)(((kd >> 2) * 1024 + (kd & 3) * 32) >> 4), idesc, kd > 0 ? 1u : 0u);
                    tc::commit(s_done + st);
                }
                __syncwarp();
            }
        }
    } else if (warp == 11) {
        // ---- O (+)= P V ---------------------------------------------------------------------
        constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) |
                                   ((uint32_t)(128 >> 4) << 24);
        const uint64_t dv = tree_desc(tc::smem_addr(sm + Ly::V), 1024, Ly::GRP);
        int it = 0, seg = 0;
        while (ok && walk.next(s)) {
            if (seg > 0 && !wait(o_free, seg - 1)) break;  // O of the segment before has been read
            ++seg;
            for (int j = s.t0; j < s.t1; ++j, ++it) {
                const int st = it & 1, steps = (keys_of(s, j) + 15) / 16;
                if (!wait(full_v + st, it >> 1) || !wait(p_ready + st, it >> 1)) break;
                tc::fence_after();
                if (tree_elect()) {
                    const uint32_t pa = tm + Ly::P_COL + st * (BK / 2);
                    const uint64_t vb = dv + ((uint32_t)(st * Ly::TILE) >> 4);
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk)
                        if (kk < steps)
                            tree_mma_ta(tm + Ly::O_COL, pa + 8 * kk, vb + (uint32_t)((2 * kk * Ly::GRP) >> 4), idesc,
                                        (j > s.t0 || kk > 0) ? 1u : 0u);
                    tc::commit(pv_done + st);
                }
                __syncwarp();
            }
        }
    } else {
        // ---- softmax and epilogue: thread = row r of the tile (TMEM lane r), of group wg ---------
        const int q4 = warp & 3, r = 32 * q4 + lane, wg = (warp - 2) >> 2;
        const uint32_t trow = tc::taddr(tm, 32 * q4, 0);
        const unsigned run_bits = (1u << nseg) - 1u;  // (at most 16 runs)
        int it = 0, tails = 0;
        // Q of the tile's rows, a row (or two of D = 128) per step, all copies in flight at once.  Rows past the
        // tree are zeros
        auto load_q = [&](const TreeSeg& t) {
            constexpr int CPR = D / 8, RPS = 32 / CPR;  // 16-byte pieces of a row, rows per step
            const int c = lane % CPR;
            int row = 32 * q4 + 16 * wg + lane / CPR, qn = (t.rt * 128 + row) / A.G, qg = (t.rt * 128 + row) % A.G;
            const __nv_bfloat16* src = A.q + ((size_t)t.first * A.Hq + t.kvh * A.G) * D + c * 8;
            const uint32_t dst = smem_u32(sm + Ly::Q + (c >> 3) * Ly::QATOM);
#pragma unroll 4
            for (int i = 0; i < 16; i += RPS, row += RPS, qg += RPS) {
                while (qg >= A.G) {
                    qg -= A.G;
                    ++qn;
                }
                const bool there = qn < t.n;
                cp_async16_or_zero(dst + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                                   there ? src + ((size_t)qn * A.Hq + qg) * D : A.q, there);
            }
            cp_async_commit();
        };
        bool have = walk.next(s);
        if (have) load_q(s);
        while (have) {
            TreeSeg after;
            const bool more = walk.next(after);
            const int node = (s.rt * 128 + r) / A.G, g = (s.rt * 128 + r) % A.G;
            const bool row_ok = node < s.n;
            const bool warp_ok = s.rt * 128 + 32 * q4 < s.n * A.G;  // a row of this warp exists
            const bool tail = s.t1 == s.nt;                         // the segment ends with the nodes' own keys
            cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready);
            float m_used = -INFINITY, l = 0.f;  // the group's sum, relative to the reference maximum it last used
            for (int j = s.t0; j < s.t1; ++j, ++it) {
                const int st = it & 1;
                if (st != wg) continue;
                const bool own_keys = j == s.nt - 1;
                wait(gone_ready + (it & 3), it >> 2);
                const unsigned gone = s_gone[it & 3] & run_bits;  // runs without keys (no page, or past the context)
                const int keys = keys_of(s, j);
                const bool full = !own_keys && gone == 0u && keys == BK;
                uint32_t seen[BK / 32];  // bit c: key c reaches this row
                if (!full) {
                    if (own_keys) {
                        wait(anc_ready + (tails & 1), tails >> 1);
                        const unsigned long long mine = row_ok ? s_anc[(tails & 3) * 64 + node] : 0ull;
#pragma unroll
                        for (int c = 0; c < BK / 32; ++c) seen[c] = c < 2 ? (uint32_t)(mine >> (32 * c)) : 0u;
                    } else {
#pragma unroll
                        for (int c = 0; c < BK / 32; ++c) {
                            const int k = keys - 32 * c;
                            seen[c] = k >= 32 ? 0xffffffffu : (k <= 0 ? 0u : (1u << k) - 1u);
                            for (int e = 0; e < 32; e += 8)  // runs are multiples of 8 keys
                                if ((gone >> ((32 * c + e) / A.R)) & 1u) seen[c] &= ~(0xffu << e);
                        }
                    }
                }
                wait(s_done + st, it >> 1);
                tc::fence_after();
                // 64 columns at a time (BK = 128: the maximum first takes the first half, which is loaded again below)
                float sv[64];
                auto load_s = [&](int half) {
                    uint32_t raw[64];
                    tc::ld32_nowait(trow + st * BK + 64 * half, raw);
                    tc::ld32_nowait(trow + st * BK + 64 * half + 32, raw + 32);
                    tc::ld_wait();
#pragma unroll
                    for (int c = 0; c < 64; ++c) sv[c] = __uint_as_float(raw[c]);
                    if (!full) {
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            sv[c] = (seen[(2 * half + (c >> 5)) % (BK / 32)] >> (c & 31)) & 1u ? sv[c] : -INFINITY;
                    }
                };
                auto top = [&]() {
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 64; ++c) mx[c & 3] = fmaxf(mx[c & 3], sv[c]);
                    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                };
                float mt = -INFINITY;
                if (warp_ok) {
#pragma unroll
                    for (int half = 0; half < BK / 64; ++half) {
                        load_s(half);
                        if (BK == 64) {  // S is in registers
                            tc::fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(s_read + st);
                        }
                        mt = fmaxf(mt, top());
                    }
                } else if (lane == 0) {
                    mbar_arrive(s_read + st);
                }
                // the reference maximum after the tile before, moved when the row's maximum passes it by more than 2^8 in
                // the exponent; the next tile's group takes it from here
                float m_ref = -INFINITY;
                if (j > s.t0) {
                    wait(decided + 4 * (wg ^ 1) + q4, (it - 1) >> 1);
                    m_ref = s_mref[r];
                }
                float f = 1.f;
                if (mt > -INFINITY && (m_ref == -INFINITY || (mt - m_ref) * A.scale_log2 > 8.f)) {
                    if (m_ref > -INFINITY) f = exp2f((m_ref - mt) * A.scale_log2);
                    m_ref = mt;
                }
                s_mref[r] = m_ref;
                __syncwarp();
                if (lane == 0) mbar_arrive(decided + 4 * wg + q4);
                if (m_ref != m_used) {
                    if (m_used > -INFINITY) l *= exp2f((m_used - m_ref) * A.scale_log2);
                    m_used = m_ref;
                }
                if (it >= 2) wait(pv_done + st, (it - 2) >> 1);  // P's buffer is free
                tc::fence_after();
                if (warp_ok) {
                    // p = 2^((s - m_ref) scale log2 e), rounded to bf16, the tensor cores' operand; the sum takes the
                    // rounded weights, like the product
                    const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref * A.scale_log2;
                    const float2 sc2 = make_float2(A.scale_log2, A.scale_log2), nm2 = make_float2(neg_m, neg_m);
#pragma unroll
                    for (int half = BK / 64 - 1; half >= 0; --half) {
                        if (half < BK / 64 - 1) {
                            load_s(half);
                            tc::fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(s_read + st);
                        }
                        float2 sum[4] = {};
                        uint32_t pk[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float2 x = __ffma2_rn(make_float2(sv[2 * e], sv[2 * e + 1]), sc2, nm2);
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(tree_ex2(x.x), tree_ex2(x.y));
                            sum[e & 3] = __fadd2_rn(sum[e & 3], __bfloat1622float2(h2));
                            pk[e] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                        l += ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) + ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
                        tree_st32(trow + Ly::P_COL + st * (BK / 2) + 32 * half, pk);
                    }
                    if (j > s.t0 && __any_sync(0xffffffffu, f != 1.f)) {  // TMEM accesses are warp-wide
                        wait(pv_done + (st ^ 1), (it - 1) >> 1);
                        tc::fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            float ov[32];
                            tc::ld32(trow + Ly::O_COL + c0, ov);
#pragma unroll
                            for (int c = 0; c < 32; ++c) ov[c] *= f;
                            tree_st32(trow + Ly::O_COL + c0, reinterpret_cast<const uint32_t*>(ov));
                        }
                    }
                    tc::st_wait();
                }
                if (!full) {
                    // a row of V without a key is cleared (up to the last step of 16), so that 0 x whatever it holds
                    // never reaches O; of the nodes' own rows the infinities and NaN are taken out too and added again
                    // at the end, for the nodes that see them.  The tile lies in order of rows, 8 at a time
                    wait(full_v + st, it >> 1);
                    uint4* vt = reinterpret_cast<uint4*>(sm + Ly::V + st * Ly::TILE);
                    const int upto = (keys + 15) / 16 * 16 * (NCH * 8);
                    const int from = own_keys || gone != 0u ? 0 : keys / 8 * (NCH * 64);
                    for (int i = from + r; i < upto; i += 128) {
                        const int row = i / (NCH * 64) * 8 + (i & 63) / 8;
                        if (row >= keys || (!own_keys && ((gone >> (row / A.R)) & 1u))) {
                            vt[i] = make_uint4(0u, 0u, 0u, 0u);
                        } else if (own_keys) {
                            const uint4 u = vt[i];
                            const uint4 x = make_uint4(nonfinite2(u.x), nonfinite2(u.y), nonfinite2(u.z), nonfinite2(u.w));
                            if (x.x | x.y | x.z | x.w) {
                                vt[i] = make_uint4(u.x & ~x.x, u.y & ~x.y, u.z & ~x.z, u.w & ~x.w);
                                atomicOr(s_bad + (tails & 3), 1ull << row);
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready + st);
            }
            // ---- the segment's O: o itself, or a part to be joined; each group has half of the columns --------
            named_bar_sync(1, 256);  // both groups are past their last tile: s_mref is final, every S is done
            const float m_ref = s_mref[r];
            if (m_used > -INFINITY && m_used != m_ref) l *= exp2f((m_used - m_ref) * A.scale_log2);
            s_l[128 * wg + r] = l;
            if (more) load_q(after);
            wait(pv_done + ((it - 1) & 1), (it - 1) >> 1);
            tc::fence_after();
            named_bar_sync(1, 256);
            l = s_l[r] + s_l[128 + r];
            unsigned long long bad = 0ull, any_bad = 0ull;
            if (tail) {
                any_bad = s_bad[tails & 3];
                bad = row_ok ? any_bad & s_anc[(tails & 3) * 64 + node] : 0ull;
                ++tails;
            }
            const bool complete = s.t0 == 0 && tail;
            const float inv = 1.f / l;  // (a row without any weight is 0 / 0)
            __nv_bfloat16* dst = A.o + ((size_t)(s.first + node) * A.Hq + s.kvh * A.G + g) * D;
            float* part = A.part + (size_t)(blockIdx.x * 2 + (s.t0 > 0 ? 0 : 1)) * (D + 2) * 128 + r;
            if (warp_ok && ok) {
#pragma unroll 1
                for (int c0 = wg * (D / 2); c0 < (wg + 1) * (D / 2); c0 += 32) {
                    float ov[32];
                    tc::ld32(trow + Ly::O_COL + c0, ov);
                    for (unsigned long long m = any_bad; m; m &= m - 1) {  // (the same for all lanes)
                        const int a = __ffsll((long long)m) - 1;
                        const uint32_t two = tree_ld1(trow + Ly::P_COL + ((it - 1) & 1) * (BK / 2) + a / 2);
                        const float p = __uint_as_float(a & 1 ? two & 0xffff0000u : two << 16);
                        const __nv_bfloat16* v = A.v_new + ((size_t)(s.first + a) * A.Hkv + s.kvh) * D + c0;
                        if ((bad >> a) & 1ull) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                const float x = __bfloat162float(v[c]);
                                if (!isfinite(x)) ov[c] = fmaf(p, x, ov[c]);
                            }
                        }
                        __syncwarp();
                    }
                    if (complete) {
                        uint4 out[4];
                        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(out);
#pragma unroll
                        for (int c = 0; c < 16; ++c) h[c] = __floats2bfloat162_rn(ov[2 * c] * inv, ov[2 * c + 1] * inv);
                        if (row_ok) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) reinterpret_cast<uint4*>(dst + c0)[c] = out[c];
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; ++c) part[(c0 + c) * 128] = ov[c];
                    }
                    __syncwarp();
                }
                if (!complete && wg == 0) {
                    part[D * 128] = m_ref;
                    part[(D + 1) * 128] = l;
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            s = after;
            have = more;
        }
    }
    tc::fence_before();
    __syncthreads();
    if (!ok && lane == 0) report_device_status(kDevWaitTimeout);
    if (warp == 1) tc::dealloc(tm, Ly::TMEM_COLS);
}

// o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the parts of a list.  Thread = row and 8 columns.  GROUPS = 4
// (few lists in many parts): four groups of threads take the parts in turn, 4 in flight at a time, and join their
// results in order; a CTA has 8 columns.  GROUPS = 1 (many lists, few parts each): a thread takes all parts, and a CTA
// has 32 columns.  Latency counts here, not bytes (the parts lie in L2).  The whole call in us, four groups against one:
// 4 lists of 38 parts 36 against 46; 256 lists, 151 of them cut, 108 against 83.
constexpr int kJoinThreads = 512;

template <int D, int GROUPS>
__global__ void __launch_bounds__(kJoinThreads, GROUPS == 4 ? 2 : 3) k_attn_tree_join(const __grid_constant__ AttnTreeArgs A) {
    constexpr int COLS = 8, DEEP = GROUPS == 4 ? 4 : 2;
    __shared__ int s_w;
    __shared__ int s_count[kJoinThreads / 32];
    __shared__ float s_part[GROUPS > 1 ? GROUPS - 1 : 1][COLS + 2][128];
    const int tid = threadIdx.x, r = tid & 127, grp = GROUPS == 4 ? tid >> 7 : 0;
    const int c0 = GROUPS == 4 ? blockIdx.y * COLS : blockIdx.y * 4 * COLS + (tid >> 7) * COLS;
    if (tid == 0) s_w = -1;
    griddep_wait();
    griddep_launch_dependents();
    // the blockIdx.x-th list that is cut: the worker that holds its second part
    static_assert(kTreeCtas <= kJoinThreads, "a thread per worker");
    const bool second = tid >= 1 && tid < A.W && A.share[2 * tid].x == tid - 1;
    const unsigned all = __ballot_sync(0xffffffffu, second);
    if ((tid & 31) == 0) s_count[tid >> 5] = __popc(all);
    __syncthreads();
    int rank = __popc(all & ((1u << (tid & 31)) - 1u));
    for (int i = 0; i < tid >> 5; ++i) rank += s_count[i];
    if (second && rank == (int)blockIdx.x) s_w = tid;
    __syncthreads();
    const int w = s_w;
    if (w < 0) return;
    const int4 list = A.share[2 * w], rows = A.share[2 * w + 1];
    const int first = w - 1, last = list.y, at = list.z * 128 + r, kvh = list.w;
    const bool there = at < rows.y * A.G;
    float M = -INFINITY, l = 0.f, o[COLS] = {};
    if (there) {
        for (int i0 = first + grp; i0 <= last; i0 += GROUPS * DEEP) {
            float m[DEEP], li[DEEP], v[DEEP][COLS];
#pragma unroll
            for (int e = 0; e < DEEP; ++e) {
                const int i = i0 + GROUPS * e;
                m[e] = -INFINITY;
                if (i > last) continue;
                // worker i's part: its share ends with the list's beginning, or begins inside it
                const float* p = A.part + (size_t)(i * 2 + (i == first ? 1 : 0)) * (D + 2) * 128 + r;
                m[e] = p[D * 128];
                li[e] = p[(D + 1) * 128];
#pragma unroll
                for (int c = 0; c < COLS; ++c) v[e][c] = p[(c0 + c) * 128];
            }
            float top = M;
#pragma unroll
            for (int e = 0; e < DEEP; ++e) top = fmaxf(top, m[e]);
            if (M > -INFINITY && top > M) {
                const float f = exp2f((M - top) * A.scale_log2);
                l *= f;
#pragma unroll
                for (int c = 0; c < COLS; ++c) o[c] *= f;
            }
            M = top;
#pragma unroll
            for (int e = 0; e < DEEP; ++e) {
                if (i0 + GROUPS * e > last) continue;
                // (a part without a key has weight 0 and zeros, or NaN where the row has no weight at all)
                const float f = m[e] == -INFINITY ? (M > -INFINITY ? 0.f : 1.f) : exp2f((m[e] - M) * A.scale_log2);
                l = fmaf(f, li[e], l);
#pragma unroll
                for (int c = 0; c < COLS; ++c) o[c] = fmaf(f, v[e][c], o[c]);
            }
        }
    }
    if (GROUPS > 1) {
        if (grp > 0) {
            s_part[grp - 1][COLS][r] = M;
            s_part[grp - 1][COLS + 1][r] = l;
#pragma unroll
            for (int c = 0; c < COLS; ++c) s_part[grp - 1][c][r] = o[c];
        }
        __syncthreads();
        if (grp > 0) return;
        float top = M;
#pragma unroll
        for (int e = 0; e < GROUPS - 1; ++e) top = fmaxf(top, s_part[e][COLS][r]);
        const float base = top == -INFINITY ? 0.f : top, f0 = M == -INFINITY && top > -INFINITY ? 0.f : exp2f((M - base) * A.scale_log2);
        l *= f0;
#pragma unroll
        for (int c = 0; c < COLS; ++c) o[c] *= f0;
#pragma unroll
        for (int e = 0; e < GROUPS - 1; ++e) {
            const float m = s_part[e][COLS][r];
            const float f = m == -INFINITY && top > -INFINITY ? 0.f : exp2f((m - base) * A.scale_log2);
            l = fmaf(f, s_part[e][COLS + 1][r], l);
#pragma unroll
            for (int c = 0; c < COLS; ++c) o[c] = fmaf(f, s_part[e][c][r], o[c]);
        }
    }
    if (!there) return;
    const float inv = 1.f / l;
    uint4 out;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&out);
#pragma unroll
    for (int c = 0; c < COLS / 2; ++c) h[c] = __floats2bfloat162_rn(o[2 * c] * inv, o[2 * c + 1] * inv);
    *reinterpret_cast<uint4*>(A.o + ((size_t)(rows.x + at / A.G) * A.Hq + kvh * A.G + at % A.G) * D + c0) = out;
}

struct TreePlan {
    int W, whole, even;
    int joins;  // most lists that can be cut
};

// sizes only: the workspace is known without a device
TreePlan tree_plan(int B, int Hq, int Hkv, int D, int max_nodes, int max_ctx) {
    const int BK = D == 256 ? 64 : 128, row_tiles = (max_nodes * (Hq / Hkv) + 127) / 128;
    const int64_t lists = (int64_t)B * Hkv * row_tiles, tiles = ((int64_t)max_ctx + BK - 1) / BK + 1;
    TreePlan p;
    p.even = lists <= kTreeCtas;
    p.whole = tiles <= kTreeWhole && p.even ? row_tiles : 0;
    p.W = p.whole ? (int)lists
                  : (int)std::min<int64_t>(kTreeCtas, std::max(lists, (lists * tiles + kTreeMinTiles - 1) / kTreeMinTiles));
    p.joins = (int)std::min<int64_t>(lists, p.W - 1);
    return p;
}

PFN_cuTensorMapEncodeTiled_v12000 tree_encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

template <int D>
cudaError_t launch_attn_tree_d(const AttnTreeJob& j, cudaStream_t st) {
    using Ly = TreeLay<D>;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = raise_smem_limit(k_attn_tree<D>, Ly::SMEM_ALLOC, smem_set);
    if (e != cudaSuccess) return e;
    PFN_cuTensorMapEncodeTiled_v12000 enc = tree_encode_fn();
    if (!enc) return cudaErrorInvalidValue;
    const TreePlan p = tree_plan(j.B, j.Hq, j.Hkv, D, j.max_nodes, j.max_ctx);
    AttnTreeArgs A;
    A.q = static_cast<const __nv_bfloat16*>(j.q);
    A.v_new = static_cast<const __nv_bfloat16*>(j.v_new);
    A.block_table = j.block_table;
    A.cu_nodes = j.cu_nodes;
    A.parents = j.parents;
    A.ctx_lens = j.ctx_lens;
    A.o = static_cast<__nv_bfloat16*>(j.o);
    A.share = p.whole || p.W == 1 ? nullptr : static_cast<int4*>(j.ws);
    A.B = j.B;
    A.Hq = j.Hq;
    A.Hkv = j.Hkv;
    A.G = j.Hq / j.Hkv;
    A.part = A.share ? reinterpret_cast<float*>(A.share + 2 * p.W) : nullptr;
    A.W = p.W;
    A.whole = p.whole;
    A.even = p.even;
    A.page = j.page;
    int R = Ly::BK;
    while (j.page % R) R >>= 1;  // rows per box: gcd(page, BK); pages hold a multiple of 8 rows
    A.R = R;
    A.max_pages = j.max_pages;
    A.n_pages = j.n_pages;
    A.n_nodes = j.n_nodes;
    A.max_nodes = j.max_nodes;
    A.max_ctx = j.max_ctx;
    A.scale_log2 = j.scale * 1.4426950408889634f;
    // A box lands as [8-row group][64-column chunk][8 rows][128 bytes], whatever the page size: one copy per run of
    // page rows, and one stride between row groups for the products
    CUtensorMap maps[4];
    for (int i = 0; i < 2; ++i) {
        const cuuint64_t dims[5] = {64, 8, (cuuint64_t)Ly::NCH, (cuuint64_t)(j.page / 8),
                                    (cuuint64_t)j.Hkv * (cuuint64_t)j.n_pages};
        const cuuint64_t strides[4] = {(cuuint64_t)D * 2, 128, (cuuint64_t)8 * D * 2, (cuuint64_t)j.page * D * 2};
        const cuuint32_t box[5] = {64, 8, (cuuint32_t)Ly::NCH, (cuuint32_t)(R / 8), 1};
        const cuuint32_t es[5] = {1, 1, 1, 1, 1};
        if (enc(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(i == 0 ? j.k_pool : j.v_pool), dims,
                strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    for (int i = 0; i < 2; ++i) {
        const cuuint64_t dims[4] = {64, (cuuint64_t)j.n_nodes, (cuuint64_t)Ly::NCH, (cuuint64_t)j.Hkv};
        const cuuint64_t strides[3] = {(cuuint64_t)j.Hkv * D * 2, 128, (cuuint64_t)D * 2};
        const cuuint32_t box[4] = {64, 8, (cuuint32_t)Ly::NCH, 1};
        const cuuint32_t es[4] = {1, 1, 1, 1};
        if (enc(&maps[2 + i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(i == 0 ? j.k_new : j.v_new), dims,
                strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    e = launch_pdl(k_attn_tree<D>, dim3((unsigned)p.W), dim3(kTreeThreads), Ly::SMEM_ALLOC, st, maps[0], maps[1],
                   maps[2], maps[3], A);
    if (e != cudaSuccess || p.whole || p.W == 1) return e;
    if (4 * p.joins >= p.W) return launch_pdl(k_attn_tree_join<D, 1>, dim3((unsigned)p.joins, D / 32), dim3(kJoinThreads), 0, st, A);
    return launch_pdl(k_attn_tree_join<D, 4>, dim3((unsigned)p.joins, D / 8), dim3(kJoinThreads), 0, st, A);
}

}  // namespace

size_t attn_tree_workspace_bytes(int B, int Hq, int Hkv, int D, int max_nodes, int max_ctx) {
    if (B == 0) return 0;
    const TreePlan p = tree_plan(B, Hq, Hkv, D, max_nodes, max_ctx);
    return p.whole || p.W == 1 ? 0 : (size_t)p.W * (32 + 2 * (D + 2) * 128 * 4);
}

cudaError_t launch_attn_tree(const AttnTreeJob& j, cudaStream_t st) {
    if (j.B == 0 || j.n_nodes == 0) return cudaSuccess;
    return j.D == 256 ? launch_attn_tree_d<256>(j, st) : launch_attn_tree_d<128>(j, st);
}

cudaError_t take_device_status_attn_tree(unsigned* out) { return take_device_status_tu(out); }

}  // namespace gdn
