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

#include "gdn_common.cuh"
#include "gdn_internal.h"
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

template <int D, typename TA>
cudaError_t launch_verify_t(const TreeArgs& A, cudaStream_t st) {
    static std::atomic<uint64_t> smem_set{0};
    const int most = tree_smem(D, kTreeMax).total;
    const cudaError_t e = raise_smem_limit(k_tree_verify<D, TA>, most, smem_set);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_tree_verify<D, TA>, dim3(A.g.Hv, A.job.B), dim3(kTreeThreads),
                      (size_t)tree_smem(D, A.nmax).total, st, A);
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
