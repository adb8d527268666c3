// gdn_tree.cu -- the gated delta rule over a tree of drafted tokens: the outputs of
// every node without writing a state (k_tree_verify), and an accepted path applied to
// the state in place (k_tree_commit).
//
// A node's state is its parent's after one token, S_i = alpha_i S_p (I - beta_i k_i k_i^T)
// + beta_i v_i k_i^T, so the states of a tree differ node by node; but all of them are
// the cached state S_0 plus rank-one terms along the node's line of ancestors.  With
// G_i = the sum of log alpha over the line (the node included) and anc(i) the line,
//   u_i = beta_i (v_i - e^{G_i} S_0 k_i - sum_{j in anc(i), j != i} e^{G_i - G_j} (k_i . k_j) u_j)
//   o_i = e^{G_i} S_0 q_i + sum_{j in anc(i)} e^{G_i - G_j} (q_i . k_j) u_j
// (the WY form of a chunk with the tree's mask in the place of the causal one).  The state is read
// once for all nodes, no state of a node is formed, and every exponent is <= 0.  This is the
// verify without snapshots of "Forge: how I wrote my own inference engine and overtook llama.cpp"
// (27 August) for drafts that branch.
#include <cooperative_groups.h>

#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_tc.cuh"
#include "gdn_tma.cuh"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

constexpr int kTreeThreads = 256;
constexpr int kTreeMax = 64;  // nodes of a tree: one bit each of a 64-bit mask

struct TreeArgs {
    Geom g;
    LayerParams p;
    TreeJob job;
    int nmax;  // nodes per tree that shared memory has room for
};

__device__ __forceinline__ float tree_warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// rows of S in shared memory are padded by 16 bytes so that 8 threads reading 16 bytes of
// 8 rows touch all banks once
__host__ __device__ inline int tree_s_stride(int D) { return D + 4; }

struct TreeSmem {
    int bar, S, k, q, u, pk, pq, sc, anc, up, total;
};

__host__ __device__ inline TreeSmem tree_smem(int D, int n) {
    auto round = [](int v) { return (v + 15) & ~15; };
    TreeSmem s;
    int o = 0;
    s.bar = o; o += 16;
    s.S = o; o += D * tree_s_stride(D) * 4;
    s.k = o; o += n * D * 4;
    s.q = o; o += n * D * 4;               // q, then o once the line sums are taken
    s.u = o; o += n * D * 4;               // v, then u
    s.pk = o; o = round(o + n * n * 4);    // e^{G_i - G_j} k_i . k_j
    s.pq = o; o = round(o + n * n * 4);    // e^{G_i - G_j} q_i . k_j
    s.sc = o; o += n * 4 * 4;              // g, beta, G, e^G per node
    s.anc = o; o += n * 8;                 // ancestors and the node itself, one bit each
    s.up = o; o = round(o + n * 4);        // parent within the tree, -1: the cached state
    s.total = o;
    return s;
}

// One CTA per (v-head, tree).  The simple form: fp32 on the CUDA cores throughout.
template <int D, typename TA>
__global__ void __launch_bounds__(kTreeThreads) k_tree_verify(const __grid_constant__ TreeArgs A) {
    using L = Act<TA>;
    const Geom& g = A.g;
    const TreeJob& J = A.job;
    const int j = blockIdx.x, h = j / g.G, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int nwarp = kTreeThreads / 32;
    const int Hk = g.Hk, Hv = g.Hv, K = g.K, Km1 = g.K - 1, C = g.C_ch;
    const bool raw = g.flags & kFlagRawQKV;
    griddep_wait();  // launched with programmatic serialization
    griddep_launch_dependents();
    const int slot = J.slot_idx[b];
    const int64_t first = J.cu_nodes[b];
    const int64_t count = (int64_t)J.cu_nodes[b + 1] - first;
    if (slot < 0 || slot >= J.n_slots || first < 0 || count < 1 || count > J.max_nodes || first + count > J.n_nodes)
        return;
    const int n = (int)count;

    extern __shared__ __align__(128) unsigned char smem[];
    const TreeSmem lay = tree_smem(D, A.nmax);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + lay.bar);
    float* S = reinterpret_cast<float*>(smem + lay.S);
    float* ks = reinterpret_cast<float*>(smem + lay.k);
    float* qs = reinterpret_cast<float*>(smem + lay.q);
    float* us = reinterpret_cast<float*>(smem + lay.u);
    float* pk = reinterpret_cast<float*>(smem + lay.pk);
    float* pq = reinterpret_cast<float*>(smem + lay.pq);
    float* sc = reinterpret_cast<float*>(smem + lay.sc);
    unsigned long long* anc = reinterpret_cast<unsigned long long*>(smem + lay.anc);
    int* up = reinterpret_cast<int*>(smem + lay.up);
    constexpr int SS = D + 4;

    // the state of (slot, j), a row at a time into padded rows
    const float* Sg = J.state_pool + ((size_t)slot * Hv + j) * D * D;
    if (tid == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(bar, D * D * 4);
        for (int r = 0; r < D; ++r) bulk_g2s(S + r * SS, Sg + (size_t)r * D, D * 4, bar);
    }
    // a parent outside [0, i) stands for the end of the cached sequence
    if (tid < n) {
        const int p = J.parents[first + tid];
        up[tid] = p >= 0 && p < tid ? p : -1;
        float gl, beta;
        gates(L::ld(J.a, (first + tid) * Hv + j), L::ld(J.b, (first + tid) * Hv + j),
              g.flags & kFlagGatesDirect ? 0.f : A.p.A_log[j],
              !(g.flags & kFlagGatesDirect) && A.p.dt_bias ? A.p.dt_bias[j] : 0.f, g.flags & kFlagGatesDirect, gl, beta);
        sc[4 * tid] = gl;
        sc[4 * tid + 1] = beta;
    }
    __syncthreads();
    if (tid < n) {  // the node's line, and the decay along it
        unsigned long long m = 0;
        float G = 0.f;
        for (int i = tid; i >= 0; i = up[i]) {
            m |= 1ull << i;
            G += sc[4 * i];
        }
        anc[tid] = m;
        sc[4 * tid + 2] = G;
        sc[4 * tid + 3] = expf(G);
    }
    // conv + SiLU of the k-head's q and k and the v-head's v
    const TA* x = static_cast<const TA*>(J.x) + first * C;
    const TA* cp = static_cast<const TA*>(J.conv_pool) + (size_t)slot * Km1 * C;
    for (int w = tid; w < 3 * D * n; w += kTreeThreads) {
        const int i = w / (3 * D), c = w % (3 * D);
        const int ch = c < D ? h * D + c : (c < 2 * D ? Hk * D + h * D + c - D : 2 * Hk * D + j * D + c - 2 * D);
        float val;
        if (raw) {
            val = L::ld(x, (size_t)i * C + ch);
        } else {
            // taps backwards along the line, then through the conv state
            float acc = A.p.conv_b ? L::ld(A.p.conv_b, ch) : 0.f;
            int at = i, row = Km1 - 1;
            for (int m = K - 1; m >= 0; --m) {
                const float xv = at >= 0 ? L::ld(x, (size_t)at * C + ch) : L::ld(cp, (size_t)(row--) * C + ch);
                acc = fmaf(L::ld(A.p.conv_w, (size_t)ch * K + m), xv, acc);
                if (at >= 0) at = up[at];
            }
            val = siluf_(acc);
        }
        (c < D ? qs : (c < 2 * D ? ks : us))[i * D + c % D] = val;
    }
    __syncthreads();
    for (int i = warp; i < n; i += nwarp) {  // L2 norms
        float sq = 0.f, sk = 0.f;
        for (int c = lane; c < D; c += 32) {
            sq = fmaf(qs[i * D + c], qs[i * D + c], sq);
            sk = fmaf(ks[i * D + c], ks[i * D + c], sk);
        }
        sq = tree_warp_sum(sq);
        sk = tree_warp_sum(sk);
        const bool nol2 = g.flags & kFlagNoL2;
        const float rq = nol2 ? g.q_scale : g.q_scale * rsqrtf(sq + g.l2_eps);
        const float rk = nol2 ? 1.f : rsqrtf(sk + g.l2_eps);
        for (int c = lane; c < D; c += 32) {
            qs[i * D + c] *= rq;
            ks[i * D + c] *= rk;
        }
    }
    __syncthreads();
    // products of a node's k and q with the k of its line, times the decay between them
    for (int w = warp; w < n * n; w += nwarp) {
        const int i = w / n, a = w % n;
        if (!((anc[i] >> a) & 1ull)) continue;
        float dk = 0.f, dq = 0.f;
        for (int c = lane; c < D; c += 32) {
            dk = fmaf(ks[i * D + c], ks[a * D + c], dk);
            dq = fmaf(qs[i * D + c], ks[a * D + c], dq);
        }
        dk = tree_warp_sum(dk);
        dq = tree_warp_sum(dq);
        if (lane == 0) {
            const float f = expf(sc[4 * i + 2] - sc[4 * a + 2]);
            pk[i * n + a] = f * dk;
            pq[i * n + a] = f * dq;
        }
    }
    bool ok = true;
    if (warp == 0) {
        ok = mbar_wait(bar, 0);
        if (!ok) mbar_wait(bar, 0);  // bounded again: let the copies in flight land
    }
    ok = __syncthreads_and(ok);
    if (!ok) {
        if (tid == 0) report_device_status(kDevWaitTimeout);
        return;
    }
    // S_0 k_i and S_0 q_i: a thread has row r of the state and every (256 / D)-th block of 4 nodes
    constexpr int NB = 4, PARTS = kTreeThreads / D;
    const int r = tid % D, part = tid / D;
    float o_first[kTreeMax / PARTS];  // e^{G_i} S_0 q_i of the thread's nodes
#pragma unroll
    for (int blk = 0; blk < kTreeMax / (NB * PARTS); ++blk) {
        const int i0 = (blk * PARTS + part) * NB;
        if (i0 < n) {
            float ak[NB] = {}, aq[NB] = {};
            for (int c = 0; c < D; c += 4) {
                const float4 s = *reinterpret_cast<const float4*>(S + r * SS + c);
#pragma unroll
                for (int e = 0; e < NB; ++e) {
                    const int i = min(i0 + e, n - 1);
                    const float4 kv = *reinterpret_cast<const float4*>(ks + i * D + c);
                    const float4 qv = *reinterpret_cast<const float4*>(qs + i * D + c);
                    ak[e] = fmaf(s.x, kv.x, fmaf(s.y, kv.y, fmaf(s.z, kv.z, fmaf(s.w, kv.w, ak[e]))));
                    aq[e] = fmaf(s.x, qv.x, fmaf(s.y, qv.y, fmaf(s.z, qv.z, fmaf(s.w, qv.w, aq[e]))));
                }
            }
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                const int i = i0 + e;
                o_first[blk * NB + e] = i < n ? aq[e] * sc[4 * i + 3] : 0.f;
                if (i < n) us[i * D + r] -= sc[4 * i + 3] * ak[e];  // v_i - e^{G_i} S_0 k_i
            }
        }
    }
    __syncthreads();  // every q has been read: its place takes o
#pragma unroll
    for (int blk = 0; blk < kTreeMax / (NB * PARTS); ++blk) {
        const int i0 = (blk * PARTS + part) * NB;
#pragma unroll
        for (int e = 0; e < NB; ++e)
            if (i0 + e < n) qs[(i0 + e) * D + r] = o_first[blk * NB + e];
    }
    __syncthreads();
    if (tid < D) {  // the line sums, in the order of the nodes: a parent comes before its children
        for (int i = 0; i < n; ++i) {
            float su = 0.f, so = 0.f;
            unsigned long long m = anc[i] & ~(1ull << i);
            while (m) {
                const int a = __ffsll((long long)m) - 1;
                m &= m - 1;
                const float ua = us[a * D + tid];
                su = fmaf(pk[i * n + a], ua, su);
                so = fmaf(pq[i * n + a], ua, so);
            }
            const float u = sc[4 * i + 1] * (us[i * D + tid] - su);
            us[i * D + tid] = u;
            qs[i * D + tid] += fmaf(pq[i * n + i], u, so);
        }
    }
    __syncthreads();
    // gated RMSNorm over the v-head, a warp per node
    const bool outnorm = !(g.flags & kFlagNoOutNorm);
    for (int i = warp; i < n; i += nwarp) {
        float ss = 0.f;
        for (int c = lane; c < D; c += 32) ss = fmaf(qs[i * D + c], qs[i * D + c], ss);
        ss = tree_warp_sum(ss);
        const float inv = rsqrtf(ss / (float)D + g.norm_eps);
        const size_t row = ((size_t)first + i) * Hv * D + (size_t)j * D;
        for (int c = lane; c < D; c += 32) {
            float y = qs[i * D + c];
            if (outnorm) y = y * inv * L::ld(A.p.norm_w, c) * siluf_(L::ld(J.z, row + c));
            L::st(J.y, row + c, y);
        }
    }
}

// ---- the same on the tensor cores (d = 128, bf16 activations) ---------------------
// One CTA per (k-head, tree): the k-head's K^ and Q^ of all nodes are made once, as the rows of one operand
// [K^; Q^] (TF32, K-major, 128-byte swizzle), and multiplied twice:
//   [K^; Q^] K^T    the products of the nodes' keys and queries with keys (M = 128, N = nm, once), and
//   S_0 [K^; Q^]^T  per v-head (M = 128 state rows, N = 2 nm), with S_0 as it lies in the pool (fp32, brought by
//                   tensor TMA 32 columns at a time; the tensor core reads its leading 10 fraction bits, as it does of
//                   K^ and Q^ rounded).
// Then a thread has a state row: its S_0 k_i and S_0 q_i come from TMEM, and it walks the nodes in order, each
// with a list of its ancestors and their two coefficients, keeping u in shared memory (its own column, no
// barrier); o takes u's place, and all warps finish the nodes' y.  TF32's 2^-11 per operand is a quarter of the
// bf16 rounding of y; the decays, sums and norms are fp32.  The phases are short and bound by latency, so the state's
// place in shared memory is kept to half a tile: two CTAs per SM up to 32 nodes.
constexpr int kVtThreads = 288;  // 8 warps and the one that drives the copies and the products
constexpr int kVtAtom = 16384;   // 128 state rows x 32 columns

struct VtSmem {
    int S, B, v, ent, gram, node, beta, taps, gate, line, up, off, bar, total;
};

// entries of a tree's nodes: a node's ancestors, rounded up to groups of 4
__host__ __device__ inline int vt_entries(int nm) { return nm * (nm - 1) / 2 + 3 * nm; }

__host__ __device__ inline VtSmem vt_smem(int nm, int bufs) {  // nm: nodes, rounded up to 16
    VtSmem s;
    int o = 0;
    s.S = o; o += 2 * kVtAtom;                // ring of state atoms
    s.B = o; o += 2 * nm * 512;               // [K^; Q^]: 4 atoms of 2 nm rows x 128 bytes
    s.v = o; o += bufs * nm * 512;            // v, then u, then o: [node][row]
    s.ent = o; o += bufs * vt_entries(nm) * 16;
    s.gram = o; o += 2 * nm * (nm + 1) * 4;
    s.node = o; o += bufs * nm * 16;          // beta, e^G, the node's own coefficient, first entry
    s.beta = o; o += nm * 8 * 4;              // per (node, v-head of the group)
    s.taps = o; o += nm * 32;                 // offsets of the conv taps' rows from x
    s.gate = o; o += nm * 8 * 4;              // log alpha, then its sum along the line
    s.line = o; o += nm * 8;
    s.up = o; o += nm * 4;
    s.off = o; o += (nm + 4) * 4;             // first entry of each node
    s.bar = o; o += 8 * 8;
    // the Gram product reads 128 rows of each atom, whatever 2 nm is: all of them lie inside the allocation
    s.total = o > s.B + 3 * 2 * nm * 128 + kVtAtom ? o : s.B + 3 * 2 * nm * 128 + kVtAtom;
    return s;
}

struct VtArgs {
    Geom g;
    LayerParams p;
    TreeJob job;
    int nm, gv, bufs;  // gv: v-heads per CTA (G, or 1 where that fills the card better)
};

__device__ __forceinline__ float vt_silu(float x) { return __fdividef(x, 1.f + __expf(-x)); }

__device__ __forceinline__ bool vt_elect() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void vt_mma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void vt_ld8(uint32_t ta, uint32_t r[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(ta));
}

__device__ __forceinline__ void vt_st1(uint32_t ta, float v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(ta), "r"(__float_as_uint(v)) : "memory");
}

// conv + SiLU of the warp's 128 channels (ch .. ch + 3 of each lane) at the nodes i0 .. i0 + 3, all loads at once.
// As v: to v[node][4 lane].  As k or q (scale != 0): L2-normalised times scale, to row row0 + node of [K^; Q^].
// One copy of this code serves every call: the phases run once per CTA, and copies in line were bound by
// instruction fetch.
__device__ __noinline__ void vt_conv(const __nv_bfloat16* x, const long long* taps, const __nv_bfloat16* conv_w,
                                     const __nv_bfloat16* conv_b, int K, int ch, int i0, int n, float* v,
                                     unsigned char* Bt, int rows, int row0, float scale, float eps) {
    const int lane = threadIdx.x & 31;
    uint2 u[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int node = min(i0 + e, n - 1);
#pragma unroll
        for (int m = 0; m < 4; ++m) u[e][m] = __ldg(reinterpret_cast<const uint2*>(x + taps[node * 4 + m] + ch));
    }
    float w[4][4], bias[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        bias[c] = conv_b ? __bfloat162float(conv_b[ch + c]) : 0.f;
#pragma unroll
        for (int m = 0; m < 4; ++m) w[m][c] = m < K ? __bfloat162float(conv_w[(size_t)(ch + c) * K + m]) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float y[4] = {bias[0], bias[1], bias[2], bias[3]};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[e][m].x));
            const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[e][m].y));
            y[0] = fmaf(w[m][0], lo.x, y[0]);
            y[1] = fmaf(w[m][1], lo.y, y[1]);
            y[2] = fmaf(w[m][2], hi.x, y[2]);
            y[3] = fmaf(w[m][3], hi.y, y[3]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = vt_silu(y[c]);
        if (scale != 0.f) {
            const float ss = tree_warp_sum(fmaf(y[0], y[0], fmaf(y[1], y[1], fmaf(y[2], y[2], y[3] * y[3]))));
            const float f = scale * rsqrtf(ss + eps);
            if (i0 + e < n) tc::st_row4(Bt, rows, row0 + i0 + e, 4 * lane, y[0] * f, y[1] * f, y[2] * f, y[3] * f);
        } else if (i0 + e < n) {
            *reinterpret_cast<float4*>(v + (i0 + e) * 128 + 4 * lane) = make_float4(y[0], y[1], y[2], y[3]);
        }
    }
}

__global__ void __launch_bounds__(kVtThreads, 2)
    k_tree_verify_tc(const __grid_constant__ CUtensorMap ts, const __grid_constant__ VtArgs A) {
    constexpr int D = 128;
    using bf = __nv_bfloat16;
    const Geom& g = A.g;
    const TreeJob& J = A.job;
    const int nm = A.nm, gv = A.gv, per_k = g.G / gv;
    const int h = blockIdx.x / per_k, j0 = h * g.G + (blockIdx.x % per_k) * gv, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hk = g.Hk, Hv = g.Hv, K = g.K, Km1 = g.K - 1, C = g.C_ch;
    griddep_wait();  // launched with programmatic serialization
    griddep_launch_dependents();
    const int slot = J.slot_idx[b];
    const int64_t first = J.cu_nodes[b];
    const int64_t count = (int64_t)J.cu_nodes[b + 1] - first;
    if (slot < 0 || slot >= J.n_slots || first < 0 || count < 1 || count > J.max_nodes || first + count > J.n_nodes)
        return;
    const int n = (int)count;

    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    const VtSmem lay = vt_smem(nm, A.bufs);
    unsigned char* Bt = sm + lay.B;
    float* gram = reinterpret_cast<float*>(sm + lay.gram);
    float* betas = reinterpret_cast<float*>(sm + lay.beta);
    long long* taps = reinterpret_cast<long long*>(sm + lay.taps);
    float* gate = reinterpret_cast<float*>(sm + lay.gate);
    unsigned long long* line = reinterpret_cast<unsigned long long*>(sm + lay.line);
    int* up = reinterpret_cast<int*>(sm + lay.up);
    int* off = reinterpret_cast<int*>(sm + lay.off);
    uint64_t *full = reinterpret_cast<uint64_t*>(sm + lay.bar), *freed = full + 2, *done = full + 4, *bar_g = full + 6;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(full + 7);
    const int tcols = nm <= 16 ? 128 : (nm <= 32 ? 256 : 512);  // products of two v-heads, then the Gram matrix
    if (tid == 0) {
        for (int i = 0; i < 7; ++i) mbar_init(full + i, 1);
        fence_mbar_init();
    }
    if (warp == 8) tc::alloc(tslot, tcols);
    // gates, parents; taps follow the parents
    if (tid < n) {
        const int p = J.parents[first + tid];
        up[tid] = p >= 0 && p < tid ? p : -1;
        line[tid] = 1ull << tid;
    }
    for (int i = tid; i < n * gv; i += kVtThreads) {
        const int node = i / gv, jj = i % gv;
        const size_t at = (size_t)(first + node) * Hv + j0 + jj;
        float gl, beta;
        gates(__bfloat162float(static_cast<const bf*>(J.a)[at]), __bfloat162float(static_cast<const bf*>(J.b)[at]),
              A.p.A_log[j0 + jj], A.p.dt_bias ? A.p.dt_bias[j0 + jj] : 0.f, false, gl, beta);
        gate[node * 8 + jj] = gl;
        betas[node * 8 + jj] = beta;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = *tslot, tgram = tm + 4 * nm;
    const bf* xb = static_cast<const bf*>(J.x) + first * C;
    const bf* cb = static_cast<const bf*>(J.conv_pool) + (size_t)slot * Km1 * C;
    if (tid < n) {  // tap K - 1 is the node, then its ancestors, then the conv state's rows from the newest on
        int at = tid, row = Km1 - 1;
        for (int t = K - 1; t >= 0; --t) {
            taps[tid * 4 + t] = at >= 0 ? (long long)at * C : (cb - xb) + (long long)(row--) * C;
            if (at >= 0) at = up[at];
        }
        for (int t = K; t < 4; ++t) taps[tid * 4 + t] = (long long)tid * C;  // (weight 0)
    }
    __syncthreads();
    // lines, and the sums of log alpha along them, by doubling: a thread has a node and v-heads jj, jj + 4
#pragma unroll 1
    for (int reach = 1; reach < n; reach <<= 1) {
        const int i = tid & 63, jj = tid >> 6;
        int p = -1, pp = -1;
        unsigned long long m = 0;
        float s0 = 0.f, s1 = 0.f;
        if (i < n && jj < 4 && (p = up[i]) >= 0) {
            pp = up[p];
            m = line[p];
            if (jj < gv) s0 = gate[p * 8 + jj];
            if (jj + 4 < gv) s1 = gate[p * 8 + jj + 4];
        }
        __syncthreads();
        if (p >= 0) {
            if (jj < gv) gate[i * 8 + jj] += s0;
            if (jj + 4 < gv) gate[i * 8 + jj + 4] += s1;
            if (jj == 0) {
                line[i] |= m;
                up[i] = pp;
            }
        }
        __syncthreads();
    }
    bool ok = true;
    if (warp == 8) {
        // ---- copies and products: the state of each v-head in 4 atoms through a ring of two ---------
        const int atoms = 4 * gv;
        auto load = [&](int a) {
            mbar_arrive_expect_tx(full + (a & 1), kVtAtom);
            tma_tile_2d(sm + lay.S + (a & 1) * kVtAtom, &ts, (a & 3) * 32, (slot * Hv + j0 + (a >> 2)) * D, full + (a & 1));
        };
        if (lane == 0) {
            load(0);
            load(1);
        }
        __syncwarp();
        named_bar_sync(2, kVtThreads);  // [K^; Q^] is there
        const uint64_t db = tc::sdesc(tc::smem_addr(Bt)), ds = tc::sdesc(tc::smem_addr(sm + lay.S));
        const uint32_t bstep = (uint32_t)(2 * nm * 128) >> 4;
        const uint32_t id_g = tc::idesc_tf32(128, nm), id_s = tc::idesc_tf32(128, 2 * nm);
        if (vt_elect()) {  // lanes are the rows of [K^; Q^] (what lies past them is never read), columns the keys
#pragma unroll 4
            for (int k = 0; k < 16; ++k)
                vt_mma(tgram, db + (k >> 2) * bstep + (k & 3) * 2, db + (k >> 2) * bstep + (k & 3) * 2, id_g, k > 0);
            tc::commit(bar_g);
        }
        __syncwarp();
#pragma unroll 1
        for (int a = 0; a < atoms && ok; ++a) {
            const int i = a >> 2;
            if ((a & 3) == 0 && i >= 2) named_bar_sync(3, 160);  // v-head i - 2 has been read out of TMEM
            ok = __all_sync(0xffffffffu, mbar_wait(full + (a & 1), (uint32_t)((a >> 1) & 1)));
            if (!ok) break;
            if (vt_elect()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    vt_mma(tm + (i & 1) * 2 * nm, ds + (uint32_t)(((a & 1) * kVtAtom) >> 4) + k * 2,
                           db + (a & 3) * bstep + k * 2, id_s, (a & 3) > 0 || k > 0);
                tc::commit(freed + (a & 1));
                if ((a & 3) == 3) tc::commit(done + (i & 1));
            }
            __syncwarp();
            if (a + 2 < atoms) {
                ok = __all_sync(0xffffffffu, mbar_wait(freed + (a & 1), (uint32_t)((a >> 1) & 1)));
                if (!ok) break;
                if (lane == 0) load(a + 2);
                __syncwarp();
            }
        }
        if (!ok) {  // let the copies in flight land (bounded again); the others' waits give up by themselves
            for (int i = 0; i < 2; ++i) mbar_wait(full + i, 0);
            if (lane == 0) report_device_status(kDevWaitTimeout);
        }
    } else {
        if (warp == 7) {  // entries before each node: scan of the numbers of proper ancestors, in groups of 4
            int base = 0;
            for (int i0 = 0; i0 < nm; i0 += 32) {
                const int i = i0 + lane;
                int c = i < n ? (__popcll(line[i]) + 2) / 4 * 4 : 0;
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, c, s);
                    if (lane >= s) c += v;
                }
                if (i < nm) off[i + 1] = base + c;
                base += __shfl_sync(0xffffffffu, c, 31);
            }
            if (lane == 0) off[0] = 0;
        }
        auto vbuf = [&](int i) { return reinterpret_cast<float*>(sm + lay.v) + (i % A.bufs) * nm * D; };
        // batches of 4 nodes: of k, q and the first v-head's v by all warps, then of the next v-heads' v
        const int batches = (n + 3) / 4;
        auto conv = [&](int what, int i, int batch) {  // what: 0 k, 1 q, 2 v of v-head j0 + i
            vt_conv(xb, taps, static_cast<const bf*>(A.p.conv_w), static_cast<const bf*>(A.p.conv_b), K,
                    (what == 0 ? (Hk + h) * D : (what == 1 ? h * D : (2 * Hk + j0 + i) * D)) + 4 * lane, 4 * batch, n,
                    vbuf(i), Bt, 2 * nm, what == 1 ? nm : 0, what == 0 ? 1.f : (what == 1 ? g.q_scale : 0.f), g.l2_eps);
        };
#pragma unroll 1
        for (int k = warp; k < 2 * batches; k += 8) conv(k & 1, 0, k >> 1);
        fence_proxy_async_smem();
        named_bar_sync(2, kVtThreads);
        // coefficients of v-head j0 + i: a thread per (node, ancestor)
        auto make_entries = [&](int i, int t0, int nt) {
            float4* ent = reinterpret_cast<float4*>(sm + lay.ent) + (i % A.bufs) * vt_entries(nm);
            float4* nd = reinterpret_cast<float4*>(sm + lay.node) + (i % A.bufs) * nm;
            const int shift = nm <= 16 ? 4 : (nm <= 32 ? 5 : 6);
#pragma unroll 1
            for (int k = tid - t0; k < n << shift; k += nt) {
                const int node = k >> shift, a = k & ((1 << shift) - 1);
                const unsigned long long m = line[node];
                if (a > node || !((m >> a) & 1ull)) continue;
                const float G = gate[node * 8 + i], beta = betas[node * 8 + i];
                const float gq = gram[(nm + node) * (nm + 1) + a];
                if (a == node) {
                    nd[node] = make_float4(beta, __expf(G), gq, 0.f);
                    // the last group is filled up with zeros times the first ancestor's u
                    const int c = __popcll(m) - 1, first_a = __ffsll((long long)m) - 1;
                    for (int e = off[node] + c; e < off[node + 1]; ++e)
                        ent[e] = make_float4(0.f, 0.f, __int_as_float(first_a * D), 0.f);
                } else {
                    const float f = __expf(G - gate[a * 8 + i]);
                    ent[off[node] + __popcll(m & ((1ull << a) - 1ull))] =
                        make_float4(beta * f * gram[node * (nm + 1) + a], f * gq, __int_as_float(a * D), 0.f);
                }
            }
        };
        if (warp < 4 && 32 * warp < 2 * nm) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar_g, 0));
            if (ok) {
                tc::fence_after();
                const int row = 32 * warp + lane;
#pragma unroll 1
                for (int c0 = 0; c0 < n; c0 += 16) {
                    uint32_t r[16];
                    vt_ld8(tc::taddr(tgram, 32 * warp, c0), r);
                    vt_ld8(tc::taddr(tgram, 32 * warp, c0 + 8), r + 8);
                    tc::ld_wait();
#pragma unroll
                    for (int c = 0; c < 16; ++c) gram[row * (nm + 1) + c0 + c] = __uint_as_float(r[c]);
                }
            }
        }
        for (int i = 0; i < gv; ++i) {
            float* v = vbuf(i);
            if (i == 0 || A.bufs == 1) {
#pragma unroll 1
                for (int k = warp; k < batches; k += 8) conv(2, i, k);
                if (i == 0) named_bar_sync(1, 256);  // the Gram matrix is there
                make_entries(i, 0, 256);
                named_bar_sync(1, 256);
            }
            if (warp < 4) {
                float* u = v + 32 * warp + lane;
                const float4* ent = reinterpret_cast<const float4*>(sm + lay.ent) + (i % A.bufs) * vt_entries(nm);
                const float4* nd = reinterpret_cast<const float4*>(sm + lay.node) + (i % A.bufs) * nm;
                const uint32_t tr = tc::taddr(tm, 32 * warp, (i & 1) * 2 * nm);
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait(done + (i & 1), (uint32_t)((i >> 1) & 1)));
                tc::fence_after();
                // w_i = beta_i (v_i - e^{G_i} S_0 k_i) in v's place
#pragma unroll 1
                for (int c0 = 0; c0 < n; c0 += 8) {
                    uint32_t rk[8];
                    vt_ld8(tr + c0, rk);
                    tc::ld_wait();
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        if (c0 + c < n) {
                            const float4 s = nd[c0 + c];
                            u[(c0 + c) * D] = s.x * (u[(c0 + c) * D] - s.y * __uint_as_float(rk[c]));
                        }
                    }
                }
                // u_i = w_i - sum of the ancestors' terms; the line's part of o_i replaces S_0 k_i
                int e = 0;
                float4 s = nd[0];
                float wi = u[0];
#pragma unroll 1
                for (int node = 0; node < n; ++node) {
                    const int end = off[node + 1], nx = min(node + 1, n - 1);
                    const float4 s_next = nd[nx];
                    const float w_next = u[nx * D];
                    float su[4] = {}, so[4] = {};
#pragma unroll 1
                    for (; e < end; e += 4) {
                        float4 k[4];
                        float ua[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) k[q] = ent[e + q];
#pragma unroll
                        for (int q = 0; q < 4; ++q) ua[q] = u[__float_as_int(k[q].z)];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            su[q] = fmaf(k[q].x, ua[q], su[q]);
                            so[q] = fmaf(k[q].y, ua[q], so[q]);
                        }
                    }
                    const float un = wi - ((su[0] + su[1]) + (su[2] + su[3]));
                    u[node * D] = un;
                    vt_st1(tr + node, fmaf(s.z, un, (so[0] + so[1]) + (so[2] + so[3])));
                    s = s_next;
                    wi = w_next;
                }
                tc::st_wait();
                // o_i in u's place (its own column: nobody else reads u)
#pragma unroll 1
                for (int c0 = 0; c0 < n; c0 += 8) {
                    uint32_t ro[8], rq[8];
                    vt_ld8(tr + c0, ro);
                    vt_ld8(tr + nm + c0, rq);
                    tc::ld_wait();
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (c0 + c < n)
                            u[(c0 + c) * D] = fmaf(nd[c0 + c].y, __uint_as_float(rq[c]), __uint_as_float(ro[c]));
                }
                tc::fence_before();
            } else if (i + 1 < gv && A.bufs == 2) {
#pragma unroll 1
                for (int k = warp - 4; k < batches; k += 4) conv(2, i + 1, k);
                make_entries(i + 1, 128, 128);
            }
            named_bar_sync(1, 256);
            if (warp < 4 && i + 2 < gv) asm volatile("bar.arrive 3, 160;" ::: "memory");  // this v-head's columns are free
            // gated RMSNorm, a warp per node, four channels to a lane
            {
                const int j = j0 + i;
                const uint2 nw = __ldg(reinterpret_cast<const uint2*>(A.p.norm_w) + lane);
                const float2 w01 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&nw.x));
                const float2 w23 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&nw.y));
#pragma unroll 1
                for (int i0 = warp; i0 < n; i0 += 32) {
                    uint2 zr[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        zr[q] = __ldg(reinterpret_cast<const uint2*>(static_cast<const bf*>(J.z) +
                                                                    ((size_t)(first + min(i0 + 8 * q, n - 1)) * Hv + j) * D) + lane);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int node = i0 + 8 * q;
                        if (node >= n) break;
                        const float4 o = *reinterpret_cast<const float4*>(v + node * D + 4 * lane);
                        const float ss = tree_warp_sum(fmaf(o.x, o.x, fmaf(o.y, o.y, fmaf(o.z, o.z, o.w * o.w))));
                        const float inv = rsqrtf(ss / (float)D + g.norm_eps);
                        const float2 z01 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&zr[q].x));
                        const float2 z23 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&zr[q].y));
                        const __nv_bfloat162 y01 = __floats2bfloat162_rn(o.x * inv * w01.x * vt_silu(z01.x),
                                                                         o.y * inv * w01.y * vt_silu(z01.y));
                        const __nv_bfloat162 y23 = __floats2bfloat162_rn(o.z * inv * w23.x * vt_silu(z23.x),
                                                                         o.w * inv * w23.y * vt_silu(z23.y));
                        uint2 out;
                        memcpy(&out.x, &y01, 4);
                        memcpy(&out.y, &y23, 4);
                        if (ok) *(reinterpret_cast<uint2*>(static_cast<bf*>(J.y) + ((size_t)(first + node) * Hv + j) * D) + lane) = out;
                    }
                }
            }
            if (i + 1 < gv && A.bufs == 1) named_bar_sync(1, 256);  // o is read: its place takes the next v
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 8) tc::dealloc(tm, tcols);
}

template <int D, typename TA>
cudaError_t launch_verify_t(const TreeArgs& A, cudaStream_t st) {
    static std::atomic<uint64_t> smem_set{0};
    const int most = tree_smem(D, kTreeMax).total;
    const cudaError_t e = raise_smem_limit(k_tree_verify<D, TA>, most, smem_set);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_tree_verify<D, TA>, dim3(A.g.Hv, A.job.B), dim3(kTreeThreads),
                      (size_t)tree_smem(D, A.nmax).total, st, A);
}

PFN_cuTensorMapEncodeTiled_v12000 vt_encode_fn() {
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

cudaError_t launch_verify_tc(const Geom& g, const LayerParams& p, const TreeJob& job, cudaStream_t st) {
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = raise_smem_limit(k_tree_verify_tc, 227 * 1024, smem_set);
    if (e != cudaSuccess) return e;
    PFN_cuTensorMapEncodeTiled_v12000 enc = vt_encode_fn();
    if (!enc) return cudaErrorInvalidValue;
    CUtensorMap map;
    const cuuint64_t dims[2] = {128, (cuuint64_t)job.n_slots * (cuuint64_t)g.Hv * 128};
    const cuuint64_t strides[1] = {512};
    const cuuint32_t box[2] = {32, 128}, es[2] = {1, 1};
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(job.state_pool), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    VtArgs A{g, p, job, (job.max_nodes + 15) / 16 * 16, g.G, 2};
    if ((long)job.B * g.Hk < sm_count()) A.gv = 1;  // few trees: a CTA per v-head
    if (A.gv == 1) A.bufs = 1;
    const int room = A.nm > 32 ? 227 * 1024 : 113 * 1024;  // two CTAs per SM (1 KB of each one's share is the system's)
    if (vt_smem(A.nm, A.bufs).total + 1024 > room) A.bufs = 1;
    return launch_pdl(k_tree_verify_tc, dim3((unsigned)(g.Hv / A.gv), (unsigned)job.B), dim3(kVtThreads),
                      (size_t)vt_smem(A.nm, A.bufs).total + 1024, st, map, A);
}

// ---- commit ---------------------------------------------------------------------
// One CTA per (v-head, sequence), a cluster per k-head.  A warp holds D / 8 state rows in registers
// through all rows of the path (a state row's update touches no other row), so the
// state is read once and written once, straight from and to HBM, and shared memory holds only
// the k, v and gates of kComRows path rows at a time.  The G CTAs of a k-head read the
// same conv rows of k, which one of them replaces: the cluster barrier stands between.
constexpr int kComRows = 16;

struct CommitArgs {
    Geom g;
    LayerParams p;
    TreeCommitJob job;
};

template <int D, typename TA>
__global__ void __launch_bounds__(kTreeThreads) k_tree_commit(const __grid_constant__ CommitArgs A) {
    using L = Act<TA>;
    constexpr int LPR = D / 4;                       // lanes of a state row, 4 floats each
    constexpr int RPI = 32 / LPR;                    // rows of one warp-wide 128-bit access
    constexpr int NA = D / (8 * RPI);                // accesses per warp: D / 8 rows
    constexpr int nwarp = kTreeThreads / 32;
    const Geom& g = A.g;
    const TreeCommitJob& J = A.job;
    const int gi = blockIdx.x, h = blockIdx.y, j = h * g.G + gi, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hk = g.Hk, Hv = g.Hv, K = g.K, Km1 = g.K - 1, C = g.C_ch;
    const bool raw = g.flags & kFlagRawQKV;
    __shared__ __align__(16) float ks[kComRows][D];
    __shared__ float vs[kComRows][D];
    __shared__ float alpha_s[kComRows], beta_s[kComRows];
    __shared__ int rows[kTreeMax];
    __shared__ int n_s;
    griddep_wait();
    griddep_launch_dependents();
    const int slot = J.slot_idx[b];
    const int64_t first = J.cu_rows[b], count = (int64_t)J.cu_rows[b + 1] - first;
    if (slot < 0 || slot >= J.n_slots || first < 0 || count < 1 || count > J.max_rows || first + count > J.n_rows)
        return;  // the whole cluster shares b
    // the rows of the path that exist, in order (64 at most: two per lane of a warp)
    if (warp == 0) {
        int src[2];
        unsigned has[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 32 * e + lane;
            src[e] = t < count ? (J.src_rows ? J.src_rows[first + t] : (int)(first + t)) : -1;
            if (src[e] >= J.n_src) src[e] = -1;
            has[e] = __ballot_sync(0xffffffffu, src[e] >= 0);
        }
        const unsigned below = (1u << lane) - 1u;
        if (src[0] >= 0) rows[__popc(has[0] & below)] = src[0];
        if (src[1] >= 0) rows[__popc(has[0]) + __popc(has[1] & below)] = src[1];
        if (lane == 0) n_s = __popc(has[0]) + __popc(has[1]);
    }
    // the warp's state rows
    float* Sg = J.state_pool + (((size_t)slot * Hv + j) * D + warp * (D / 8)) * D;
    const int rsub = lane / LPR, col = (lane % LPR) * 4;
    float4 s[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) s[i] = *reinterpret_cast<const float4*>(Sg + (size_t)(i * RPI + rsub) * D + col);
    __syncthreads();
    const int n = n_s;
    if (n == 0) return;  // no row that exists (the whole cluster)
    const TA* x = static_cast<const TA*>(J.x);
    TA* cp = static_cast<TA*>(J.conv_pool) + (size_t)slot * Km1 * C;
    // raw input p of the sequence: the conv state's rows, then the path's
    auto hist = [&](int p, int ch) -> TA { return p < Km1 ? cp[(size_t)p * C + ch] : x[(size_t)rows[p - Km1] * C + ch]; };
    for (int t0 = 0; t0 < n; t0 += kComRows) {
        const int m = min(kComRows, n - t0);
        for (int w = tid; w < 2 * D * m; w += kTreeThreads) {
            const int t = w / (2 * D), c = w % (2 * D);
            const int ch = c < D ? Hk * D + h * D + c : 2 * Hk * D + j * D + c - D;
            float val;
            if (raw) {
                val = L::ld(x, (size_t)rows[t0 + t] * C + ch);
            } else {
                float acc = A.p.conv_b ? L::ld(A.p.conv_b, ch) : 0.f;
                for (int e = 0; e < K; ++e) {
                    const TA xv = hist(t0 + t + e, ch);
                    acc = fmaf(L::ld(A.p.conv_w, (size_t)ch * K + e), L::ld(&xv, 0), acc);
                }
                val = siluf_(acc);
            }
            if (c < D) ks[t][c] = val;
            else vs[t][c - D] = val;
        }
        if (tid < m) {
            float gl, beta;
            const size_t at = (size_t)rows[t0 + tid] * Hv + j;
            const bool direct = g.flags & kFlagGatesDirect;
            gates(L::ld(J.a, at), L::ld(J.b, at), direct ? 0.f : A.p.A_log[j],
                  !direct && A.p.dt_bias ? A.p.dt_bias[j] : 0.f, direct, gl, beta);
            alpha_s[tid] = expf(gl);
            beta_s[tid] = beta;
        }
        __syncthreads();
        if (!(g.flags & kFlagNoL2)) {
            for (int t = warp; t < m; t += nwarp) {
                float sk = 0.f;
                for (int c = lane; c < D; c += 32) sk = fmaf(ks[t][c], ks[t][c], sk);
                const float rk = rsqrtf(tree_warp_sum(sk) + g.l2_eps);
                for (int c = lane; c < D; c += 32) ks[t][c] *= rk;
            }
            __syncthreads();
        }
        for (int t = 0; t < m; ++t) {
            const float4 kv = *reinterpret_cast<const float4*>(&ks[t][col]);
            const float alpha = alpha_s[t], beta = beta_s[t];
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                float d = fmaf(s[i].x, kv.x, fmaf(s[i].y, kv.y, fmaf(s[i].z, kv.z, s[i].w * kv.w)));
#pragma unroll
                for (int off = LPR / 2; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
                const float be = beta * (vs[t][warp * (D / 8) + i * RPI + rsub] - alpha * d);
                s[i].x = fmaf(alpha, s[i].x, be * kv.x);
                s[i].y = fmaf(alpha, s[i].y, be * kv.y);
                s[i].z = fmaf(alpha, s[i].z, be * kv.z);
                s[i].w = fmaf(alpha, s[i].w, be * kv.w);
            }
        }
        __syncthreads();  // ks and vs are read
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) *reinterpret_cast<float4*>(Sg + (size_t)(i * RPI + rsub) * D + col) = s[i];
    // the new conv state: the last K - 1 raw inputs, bit for bit.  A thread reads a channel's
    // inputs before it writes them; the k-head's k channels are read by the cluster's other
    // CTAs above, its q channels by none
    cg::this_cluster().sync();
    for (int c = tid; c < 3 * D; c += kTreeThreads) {
        if (c < 2 * D && c % g.G != gi) continue;
        const int ch = c < D ? h * D + c : (c < 2 * D ? Hk * D + h * D + c - D : 2 * Hk * D + j * D + c - 2 * D);
        TA v[3];
#pragma unroll
        for (int m = 0; m < 3; ++m)
            if (m < Km1) v[m] = hist(n + m, ch);
#pragma unroll
        for (int m = 0; m < 3; ++m)
            if (m < Km1) cp[(size_t)m * C + ch] = v[m];
    }
}

template <int D, typename TA>
cudaError_t launch_commit_t(const CommitArgs& A, cudaStream_t st) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)A.g.G;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)A.g.G, (unsigned)A.g.Hk, (unsigned)A.job.B);
    cfg.blockDim = dim3(kTreeThreads);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_tree_commit<D, TA>, A);
}

}  // namespace

#define GDN_BY_TYPE(FN)                                                             \
    if (g.act_bf16) {                                                               \
        switch (g.D) {                                                              \
            case 32: return FN<32, __nv_bfloat16>(A, st);                           \
            case 64: return FN<64, __nv_bfloat16>(A, st);                           \
            case 128: return FN<128, __nv_bfloat16>(A, st);                         \
        }                                                                           \
    } else {                                                                        \
        switch (g.D) {                                                              \
            case 32: return FN<32, float>(A, st);                                   \
            case 64: return FN<64, float>(A, st);                                   \
            case 128: return FN<128, float>(A, st);                                 \
        }                                                                           \
    }                                                                               \
    return cudaErrorInvalidValue

cudaError_t launch_tree_verify(const Geom& g, const LayerParams& p, const TreeJob& job, cudaStream_t st) {
    if (job.B == 0 || job.n_nodes == 0) return cudaSuccess;
    if (g.D == 128 && g.act_bf16 && g.flags == 0) {
        return launch_verify_tc(g, p, job, st);
    }
    const TreeArgs A{g, p, job, job.max_nodes};
    GDN_BY_TYPE(launch_verify_t);
}

cudaError_t launch_tree_commit(const Geom& g, const LayerParams& p, const TreeCommitJob& job, cudaStream_t st) {
    if (job.B == 0 || job.n_rows == 0) return cudaSuccess;
    const CommitArgs A{g, p, job};
    GDN_BY_TYPE(launch_commit_t);
}

cudaError_t take_device_status_tree(unsigned* out) { return take_device_status_tu(out); }

}  // namespace gdn
