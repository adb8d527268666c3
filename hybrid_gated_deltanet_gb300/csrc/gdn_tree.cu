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

#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_tc.cuh"
#include "gdn_tma.cuh"


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

// NV values per lane (a power of two, at most 8), summed over groups of 8 lanes; lane l of a group ends with value
// l / (8 / NV): each step halves the values by exchanging the half that the partner keeps
template <int NV>
__device__ __forceinline__ float tree_sum8(float v[NV], int lane) {
    int count = NV;
#pragma unroll
    for (int s = 4; s >= 1; s >>= 1) {
        if (count > 1) {
            const bool upper = lane & s;
            count /= 2;
#pragma unroll
            for (int i = 0; i < NV / 2; ++i) {
                if (i < count) {
                    const float send = upper ? v[i] : v[i + count];
                    const float keep = upper ? v[i + count] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], s);
        }
    }
    return v[0];
}

// four consecutive activations as fp32
__device__ __forceinline__ float4 tree_ld4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 tree_ld4(const __nv_bfloat16* p) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
// acc + a . b on the paired fp32 instructions
__device__ __forceinline__ float2 tree_dot(const float4& a, const float4& b, float2 acc) {
    return __ffma2_rn(make_float2(a.z, a.w), make_float2(b.z, b.w), __ffma2_rn(make_float2(a.x, a.y), make_float2(b.x, b.y), acc));
}
__device__ __forceinline__ void tree_prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// x sigmoid(x) by the SFU's exponential and reciprocal, five instructions (the functions of the math library spend as many
// again on subnormal arguments, which the sum with 1 absorbs here): 2^-21 relative at the sizes of a conv's outputs
__device__ __forceinline__ float tree_silu(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return x * r;
}

// entries of a tree's nodes: a node's proper ancestors, rounded up to groups of 4
__host__ __device__ inline int tree_entries(int n) { return n * (n - 1) / 2 + 3 * n; }

struct TreeSmem {
    int k, q, u, p, r, w, ent, node, anc, up, off, taps, total;
};

__host__ __device__ inline TreeSmem tree_smem(int D, int n) {
    auto round = [](int v) { return (v + 15) & ~15; };
    TreeSmem s;
    int o = 0;
    s.k = o; o += n * D * 4;
    s.q = o; o += n * D * 4;
    s.u = o; o += n * D * 4;                      // v, then u
    s.p = o; o += n * D * 4;                      // S_0 k_i
    s.r = o; o += n * D * 4;                      // S_0 q_i, then o
    s.w = s.p;                                    // conv weights [q, k, v][4 taps][D] (12 rows) and bias [3][D], till p is made
    if (n < 8) o += (8 - n) * 2 * D * 4;          // (15 rows in p's and r's place)
    s.ent = o; o += tree_entries(n) * 16;         // per (node, proper ancestor): two coefficients and the ancestor
    s.node = o; o += n * 16;                      // beta, G, e^G, q_i . k_i
    s.anc = o; o += n * 8;                        // ancestors and the node itself, one bit each
    s.up = o; o += n * 4;                         // parent within the tree, -1: the cached state
    s.off = o; o = round(o + (n + 1) * 4);        // first entry of each node
    s.taps = o; o += n * 16;                      // rows of the conv taps: a node, or 64 + a row of the conv state
    s.total = o;
    return s;
}

// One CTA per (v-head, tree), fp32 on the CUDA cores throughout: fp32 activations, d < 128 and the flags.  A
// warp has d / 8 state rows in registers, 8 lanes to a row, and takes the nodes' k and q one after another; the sums
// of its dot products are reduced together (7 shuffles for 8 of them).  Bound by instructions: 4 d^2 multiply-adds per
// node against 4 d^2 bytes of state per tree, and as much again for the shuffles, the conv and the line sums.
template <int D, typename TA>
__global__ void __launch_bounds__(kTreeThreads, 2) k_tree_verify(const __grid_constant__ TreeArgs A) {
    using L = Act<TA>;
    constexpr int LPN = D / 4, NPW = 32 / LPN;  // lanes of a node's channels, nodes of a warp (conv, output)
    constexpr int RL = D / 32;                  // state rows and 4-column chunks of a lane
    constexpr int nwarp = kTreeThreads / 32;
    const Geom& g = A.g;
    const TreeJob& J = A.job;
    const int j = blockIdx.x, h = j / g.G, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hk = g.Hk, Hv = g.Hv, K = g.K, Km1 = g.K - 1, C = g.C_ch;
    const bool raw = g.flags & kFlagRawQKV, direct = g.flags & kFlagGatesDirect;
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
    float* ks = reinterpret_cast<float*>(smem + lay.k);
    float* qs = reinterpret_cast<float*>(smem + lay.q);
    float* us = reinterpret_cast<float*>(smem + lay.u);
    float* ps = reinterpret_cast<float*>(smem + lay.p);
    float* rs = reinterpret_cast<float*>(smem + lay.r);
    float* ws = reinterpret_cast<float*>(smem + lay.w);
    float4* ent = reinterpret_cast<float4*>(smem + lay.ent);
    float4* nd = reinterpret_cast<float4*>(smem + lay.node);
    unsigned long long* anc = reinterpret_cast<unsigned long long*>(smem + lay.anc);
    int* up = reinterpret_cast<int*>(smem + lay.up);
    int* off = reinterpret_cast<int*>(smem + lay.off);
    int* taps = reinterpret_cast<int*>(smem + lay.taps);

    // the state on its way to L2 while the inputs are prepared
    const float* Sg = J.state_pool + ((size_t)slot * Hv + j) * D * D;
    for (int i = tid; i < D * D / 32; i += kTreeThreads) tree_prefetch(Sg + i * 32);
    // a parent outside [0, i) stands for the end of the cached sequence
    float gl = 0.f, beta = 0.f;
    if (tid < n) {
        const int p = J.parents[first + tid];
        up[tid] = p >= 0 && p < tid ? p : -1;
        gates(L::ld(J.a, (first + tid) * Hv + j), L::ld(J.b, (first + tid) * Hv + j), direct ? 0.f : A.p.A_log[j],
              !direct && A.p.dt_bias ? A.p.dt_bias[j] : 0.f, direct, gl, beta);
        nd[tid] = make_float4(beta, gl, 0.f, 0.f);
    }
    auto channel = [&](int kind) { return (kind == 0 ? h : (kind == 1 ? Hk + h : 2 * Hk + j)) * D; };
    if (!raw) {
        for (int i = tid; i < 3 * D; i += kTreeThreads) {
            const int ch = channel(i / D) + i % D;
#pragma unroll
            for (int t = 0; t < 4; ++t) {  // (taps are aligned at the newest)
                const int m = t - (4 - K);
                ws[(i / D * 4 + t) * D + i % D] = m >= 0 ? L::ld(A.p.conv_w, (size_t)ch * K + m) : 0.f;
            }
            ws[12 * D + i] = A.p.conv_b ? L::ld(A.p.conv_b, ch) : 0.f;
        }
    }
    __syncthreads();
    float G = 0.f;
    if (tid < n) {  // the node's line, and the decay along it
        unsigned long long m = 0;
        for (int i = tid; i >= 0; i = up[i]) {
            m |= 1ull << i;
            G += nd[i].y;
        }
        anc[tid] = m;
    } else if (tid >= 128 && tid - 128 < n) {
        // its conv taps: the last is the node, then its ancestors, then the conv state, newest first
        const int i = tid - 128;
        int at = i, row = Km1 - 1;
        for (int t = 3; t >= 0; --t) {
            const bool live = 3 - t < K;
            taps[i * 4 + t] = !live ? i : (at >= 0 ? at : 64 + row--);
            if (live && at >= 0) at = up[at];
        }
    }
    __syncthreads();
    if (tid < n) nd[tid] = make_float4(beta, G, expf(G), 0.f);
    if (warp == nwarp - 1) {  // entries before each node
        int base = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            int c = i < n ? (__popcll(anc[i]) + 2) / 4 * 4 : 0;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, c, s);
                if (lane >= s) c += v;
            }
            if (i < n) off[i + 1] = base + c;
            base += __shfl_sync(0xffffffffu, c, 31);
        }
        if (lane == 0) off[0] = 0;
    }
    // conv + SiLU, then the L2 norm, of q (kind 0), k (1) and v (2): a warp takes NB x NPW nodes at a time
    const TA* x = static_cast<const TA*>(J.x) + first * C;
    const TA* cp = static_cast<const TA*>(J.conv_pool) + (size_t)slot * Km1 * C;
    {
        constexpr int NB = 3;
        const int sub = lane / LPN, c4 = (lane % LPN) * 4, groups = (n + NB * NPW - 1) / (NB * NPW);
#pragma unroll 1
        for (int unit = warp; unit < 3 * groups; unit += nwarp) {
            const int kind = unit / groups, i0 = unit % groups * NB * NPW + sub, ch = channel(kind) + c4;
            float4 v[NB][4];
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                const int i = min(i0 + e * NPW, n - 1);
                const int4 t4 = *reinterpret_cast<const int4*>(taps + i * 4);
                const int tap[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int at = raw ? i : tap[t];
                    v[e][t] = tree_ld4(at < 64 ? x + (size_t)at * C + ch : cp + (size_t)(at - 64) * C + ch);
                }
            }
            float y[NB][4], ss[NB];
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                if (raw) {
                    y[e][0] = v[e][3].x, y[e][1] = v[e][3].y, y[e][2] = v[e][3].z, y[e][3] = v[e][3].w;
                } else {
                    const float4 bias = *reinterpret_cast<const float4*>(ws + 12 * D + kind * D + c4);
                    y[e][0] = bias.x, y[e][1] = bias.y, y[e][2] = bias.z, y[e][3] = bias.w;
                }
            }
            if (!raw) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (t < 4 - K) continue;
                    const float4 w = *reinterpret_cast<const float4*>(ws + (kind * 4 + t) * D + c4);
#pragma unroll
                    for (int e = 0; e < NB; ++e) {
                        y[e][0] = fmaf(w.x, v[e][t].x, y[e][0]);
                        y[e][1] = fmaf(w.y, v[e][t].y, y[e][1]);
                        y[e][2] = fmaf(w.z, v[e][t].z, y[e][2]);
                        y[e][3] = fmaf(w.w, v[e][t].w, y[e][3]);
                    }
                }
#pragma unroll
                for (int e = 0; e < NB; ++e)
#pragma unroll
                    for (int c = 0; c < 4; ++c) y[e][c] = tree_silu(y[e][c]);
            }
#pragma unroll
            for (int e = 0; e < NB; ++e)
                ss[e] = fmaf(y[e][0], y[e][0], fmaf(y[e][1], y[e][1], fmaf(y[e][2], y[e][2], y[e][3] * y[e][3])));
            if (kind < 2) {
#pragma unroll
                for (int o = LPN / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int e = 0; e < NB; ++e) ss[e] += __shfl_xor_sync(0xffffffffu, ss[e], o);
            }
            float* to = (kind == 0 ? qs : (kind == 1 ? ks : us)) + c4;
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                float f = kind < 2 && !(g.flags & kFlagNoL2) ? rsqrtf(ss[e] + g.l2_eps) : 1.f;
                if (kind == 0) f *= g.q_scale;
                if (i0 + e * NPW < n)
                    *reinterpret_cast<float4*>(to + (i0 + e * NPW) * D) = make_float4(y[e][0] * f, y[e][1] * f, y[e][2] * f, y[e][3] * f);
            }
        }
    }
    // the warp's state rows: row rl * 4 + group, columns 4 l8 + 32 c of lane l8 of the group
    const int l8 = lane & 7, grp = lane >> 3, row0 = warp * (D / 8) + grp;
    float4 S[RL][RL];
#pragma unroll
    for (int r = 0; r < RL; ++r)
#pragma unroll
        for (int c = 0; c < RL; ++c)
            S[r][c] = __ldg(reinterpret_cast<const float4*>(Sg + (size_t)(row0 + r * 4) * D + 4 * l8 + 32 * c));
    __syncthreads();
    // a node's products with the keys of its line, times the decay between them: a warp per node, 8 lanes per ancestor
    for (int i = warp; i < n; i += nwarp) {
        const float4 me = nd[i];
        unsigned long long m = anc[i];
        const int first_a = __ffsll((long long)m) - 1, start = off[i];
        for (int at = 0; m; at += 4) {
            int a = i;  // (the node itself again past the end)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e == grp && m) a = __ffsll((long long)m) - 1;
                m &= m - 1;
            }
            float2 dk = make_float2(0.f, 0.f), dq = dk;
#pragma unroll
            for (int c = 0; c < RL; ++c) {
                const float4 ka = *reinterpret_cast<const float4*>(ks + a * D + 4 * l8 + 32 * c);
                dk = tree_dot(*reinterpret_cast<const float4*>(ks + i * D + 4 * l8 + 32 * c), ka, dk);
                dq = tree_dot(*reinterpret_cast<const float4*>(qs + i * D + 4 * l8 + 32 * c), ka, dq);
            }
            float v[2] = {dk.x + dk.y, dq.x + dq.y};
            const float t = tree_sum8<2>(v, lane), q1 = __shfl_down_sync(0xffffffffu, t, 4);  // lane 0 of a group: k; lane 4: q
            if (l8 == 0) {
                if (a == i) {
                    nd[i].w = q1;
                } else {
                    const float f = expf(me.y - nd[a].y);
                    ent[start + at + grp] = make_float4(me.x * f * t, f * q1, __int_as_float(a * D), 0.f);
                }
            }
        }
        // the last group is filled up with zeros times the first ancestor's u
        const int c = __popcll(anc[i]) - 1;
        if (lane < off[i + 1] - start - c) ent[start + c + lane] = make_float4(0.f, 0.f, __int_as_float(first_a * D), 0.f);
    }
    // S_0 k_i and S_0 q_i of the warp's rows (ps and rs replace the conv weights: everybody is past them)
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        float2 d[2 * RL];
#pragma unroll
        for (int r = 0; r < 2 * RL; ++r) d[r] = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < RL; ++c) {
            const float4 kv = *reinterpret_cast<const float4*>(ks + i * D + 4 * l8 + 32 * c);
            const float4 qv = *reinterpret_cast<const float4*>(qs + i * D + 4 * l8 + 32 * c);
#pragma unroll
            for (int r = 0; r < RL; ++r) {
                d[2 * r] = tree_dot(S[r][c], kv, d[2 * r]);
                d[2 * r + 1] = tree_dot(S[r][c], qv, d[2 * r + 1]);
            }
        }
        float v[2 * RL];
#pragma unroll
        for (int r = 0; r < 2 * RL; ++r) v[r] = d[r].x + d[r].y;
        const float t = tree_sum8<2 * RL>(v, lane);
        const int which = l8 / (4 / RL);  // the lane's value: row which / 2, with k or q
        if (l8 % (4 / RL) == 0) ((which & 1) ? rs : ps)[i * D + row0 + (which >> 1) * 4] = t;
    }
    __syncthreads();
    if (tid < D / 2) {  // thread = two state rows: u and o, in the order of the nodes (a parent comes before its children)
        float2* u = reinterpret_cast<float2*>(us) + tid;
        constexpr int H = D / 2;
        int e = 0;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const float4 s = nd[i];
            const int end = off[i + 1];
            const float2 p = reinterpret_cast<const float2*>(ps)[i * H + tid], r = reinterpret_cast<const float2*>(rs)[i * H + tid];
            const float2 v = u[i * H];
            float2 su[2] = {}, so[2] = {};
#pragma unroll 1
            for (; e < end; e += 4) {
                float4 c[4];
                float2 ua[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) c[q] = ent[e + q];
#pragma unroll
                for (int q = 0; q < 4; ++q) ua[q] = u[__float_as_int(c[q].z) / 2];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    su[q & 1] = __ffma2_rn(make_float2(c[q].x, c[q].x), ua[q], su[q & 1]);
                    so[q & 1] = __ffma2_rn(make_float2(c[q].y, c[q].y), ua[q], so[q & 1]);
                }
            }
            const float2 un = make_float2(s.x * (v.x - s.z * p.x) - (su[0].x + su[1].x), s.x * (v.y - s.z * p.y) - (su[0].y + su[1].y));
            u[i * H] = un;
            reinterpret_cast<float2*>(rs)[i * H + tid] =
                make_float2(fmaf(s.w, un.x, fmaf(s.z, r.x, so[0].x + so[1].x)), fmaf(s.w, un.y, fmaf(s.z, r.y, so[0].y + so[1].y)));
        }
    }
    __syncthreads();
    // gated RMSNorm over the v-head, an LPN-lane group per node
    const bool outnorm = !(g.flags & kFlagNoOutNorm);
    const int sub = lane / LPN, c4 = (lane % LPN) * 4;
    float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
    if (outnorm) w = tree_ld4(static_cast<const TA*>(A.p.norm_w) + c4);
#pragma unroll 2
    for (int i0 = warp * NPW + sub; i0 - sub < n; i0 += nwarp * NPW) {
        const int i = min(i0, n - 1);
        const size_t row = ((size_t)first + i) * Hv * D + (size_t)j * D + c4;
        float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        if (outnorm) z = tree_ld4(static_cast<const TA*>(J.z) + row);
        const float4 o = *reinterpret_cast<const float4*>(rs + i * D + c4);
        float ss = fmaf(o.x, o.x, fmaf(o.y, o.y, fmaf(o.z, o.z, o.w * o.w)));
#pragma unroll
        for (int s = LPN / 2; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
        float y[4] = {o.x, o.y, o.z, o.w};
        if (outnorm) {
            const float inv = rsqrtf(ss / (float)D + g.norm_eps);
            y[0] *= inv * w.x * tree_silu(z.x);
            y[1] *= inv * w.y * tree_silu(z.y);
            y[2] *= inv * w.z * tree_silu(z.z);
            y[3] *= inv * w.w * tree_silu(z.w);
        }
        if (i0 < n) {
#pragma unroll
            for (int c = 0; c < 4; ++c) L::st(J.y, row + c, y[c]);
        }
    }
}

// ---- the same on the tensor cores (d = 128, bf16 activations) ---------------------
// One CTA per (k-head, tree).  With p_j = S_0 k_j, r_j = S_0 q_j and w_j = beta_j (v_j - e^{G_j} p_j), the sums above
// are linear in w: u = T w with T the inverse of the unit triangular matrix of the ancestors' coefficients, and
//   o_i = e^{G_i} r_i + sum_j M_ij w_j,   M = (the queries' coefficients) T,
// with M of n x n per v-head and the same for all 128 state rows.  So (all products TF32, fp32 accumulation):
//   [K^; Q^] K^T    M = 128, N = nm, once: the products of the nodes' keys and queries with keys;
//   S_0 [K^; Q^]^T  per v-head, M = 128 state rows, N = 2 nm, S_0 as it lies in the pool (fp32, brought by tensor
//                   TMA 32 columns at a time; the tensor core reads its leading 10 fraction bits, as it does of K^ and
//                   Q^ rounded): p and r in TMEM;
//   r += w M^T      w in TMEM in p's place.
// M comes from one warp (two above 32 nodes), a lane per column of T, walking the nodes in order with the
// coefficients of each node's line; it runs ahead of the other warps, which make v, w, o and y.  TF32's 2^-11 per
// operand is a quarter of the bf16 rounding of y; the decays, T's sums and the norms are fp32.  The phases are short
// and bound by latency and instructions, so the state's place in shared memory is kept to half a tile: two CTAs
// per SM up to 32 nodes.
constexpr int kVtThreads = 288;  // 8 warps and the one that drives the copies and the products
constexpr int kVtAtom = 16384;   // 128 state rows x 32 columns

struct VtSmem {
    int S, B, M, v, gram, ent, who, w, own, taps, gate, beta, eg, line, up, off, bar, total;
};

// entries of a tree's nodes: a node's proper ancestors, rounded up to pairs
__host__ __device__ inline int vt_entries(int nm) { return nm * (nm - 1) / 2 + nm; }

__host__ __device__ inline VtSmem vt_smem(int nm, int gv) {  // nm: nodes, rounded up to 16
    const int halves = (nm + 31) / 32, two = gv > 1 ? 2 : 1;   // v-heads are taken two at a time
    VtSmem s;
    int o = 0;
    s.S = o; o += 2 * kVtAtom;               // ring of state atoms
    s.B = o; o += 2 * nm * 512;              // [K^; Q^]: 4 atoms of 2 nm rows x 128 bytes
    s.M = o; o += two * halves * nm * 128;   // M of two v-heads: atoms of nm rows x 32 columns
    s.v = o; o += nm * 512;                  // v, then o: [node][row]; at first, from M on: raw q, k of [K - 1 + n] rows
    if (o < s.M + (nm + 3) * 512) o = s.M + (nm + 3) * 512;
    s.gram = o;                              // the products of the nodes' k and q with keys; then T: [v-head][half][node][32]
    o += 2 * nm * (nm + 1) * 4 > two * halves * nm * 128 ? 2 * nm * (nm + 1) * 4 : two * halves * nm * 128;
    s.ent = o; o += two * vt_entries(nm) * 8;         // two coefficients per (node, proper ancestor)
    s.who = o; o += (vt_entries(nm) + 15) / 16 * 16;  // and that ancestor
    s.w = o; o += (2 + two) * 4 * 128 * 2;   // conv weights of k, q and two v-heads: [4 taps][128]
    s.own = o; o += nm * 4;                  // q_i . k_i
    s.taps = o; o += nm * 16;                // rows of the conv taps: a node, or 64 + a row of the conv state
    s.gate = o; o += nm * gv * 4;            // log alpha, then its sum G along the line, per (node, v-head)
    s.beta = o; o += nm * gv * 4;
    s.eg = o; o += nm * gv * 4;              // e^G
    s.line = o; o += nm * 8;
    s.up = o; o += nm * 4;
    s.off = o; o += (nm + 4) * 4;            // first entry of each node
    s.bar = o; o += 16 * 8;
    // the Gram product reads 128 rows of each atom, whatever 2 nm is: all of them lie inside the allocation
    s.total = o > s.B + 3 * 2 * nm * 128 + kVtAtom ? o : s.B + 3 * 2 * nm * 128 + kVtAtom;
    return s;
}

struct VtArgs {
    Geom g;
    LayerParams p;
    TreeJob job;
    int nm, gv;  // gv: v-heads per CTA (G, or 1 where that fills the card better)
};

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

__device__ __forceinline__ void vt_st8(uint32_t ta, const float v[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(ta),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}

// a product with A in TMEM (lane = row, column = k)
__device__ __forceinline__ void vt_mma_ta(uint32_t d, uint32_t a, uint64_t bd, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, 1, 0;\n"
        " tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(bd), "r"(idesc)
        : "memory");
}

// warp-wide bounded wait that lets the hardware park the warp (a spin would take issue slots from the others)
__device__ __forceinline__ bool vt_wait(uint64_t* bar, int phase) {
    const uint32_t addr = smem_u32(bar);
    long long t0 = 0;
    for (int i = 0;; ++i) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(done)
            : "r"(addr), "r"((uint32_t)(phase & 1)), "r"(20000)  // up to 20 us at a time
            : "memory");
        if (__all_sync(0xffffffffu, done)) return true;
        const long long t = clock64();
        if (i == 0) t0 = t;
        if (__any_sync(0xffffffffu, t - t0 > kWaitLimitCycles)) return false;
    }
}

// two bf16 as fp32
__device__ __forceinline__ float2 vt_two(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// conv + SiLU of the warp's 128 channels (4 to a lane) at the nodes i0 .. i0 + 3, all loads at once.  `raw` != 0: k or q,
// its inputs in shared memory from there on (conv state first, 512 bytes to a row), L2-normalised times scale, to row
// row0 + node of [K^; Q^].  Else v, inputs in global memory, to v[node][4 lane].  One copy of this code serves every
// call: the phases run once per CTA, and copies in line were bound by instruction fetch.
__device__ __noinline__ void vt_conv(uint32_t raw, const unsigned char* x, const unsigned char* state, uint32_t row_bytes,
                                     const int4* taps, const uint2* w, const __nv_bfloat16* bias, int K, int i0, int n,
                                     float* v, unsigned char* Bt, int rows, int row0, float scale, float eps) {
    const int lane = threadIdx.x & 31;
    uint2 u[4][4];
    if (raw) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int4 t4 = taps[min(i0 + e, n - 1)];
            const int tap[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t at = raw + (tap[m] < 64 ? tap[m] + K - 1 : tap[m] - 64) * 512;
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(u[e][m].x), "=r"(u[e][m].y) : "r"(at));
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int4 t4 = taps[min(i0 + e, n - 1)];
            const int tap[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
            for (int m = 0; m < 4; ++m)
                u[e][m] = __ldg(reinterpret_cast<const uint2*>((tap[m] < 64 ? x : state) + (uint64_t)(tap[m] & 63) * row_bytes));
        }
    }
    float2 y[4][2];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < 2; ++c)
            y[e][c] = bias ? vt_two(reinterpret_cast<const uint32_t*>(bias)[c]) : make_float2(0.f, 0.f);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if (m < 4 - K) continue;  // a tap that d_conv < 4 does not have
        const uint2 wm = w[m * 32 + lane];
        const float2 w01 = vt_two(wm.x), w23 = vt_two(wm.y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e][0] = __ffma2_rn(w01, vt_two(u[e][m].x), y[e][0]);
            y[e][1] = __ffma2_rn(w23, vt_two(u[e][m].y), y[e][1]);
        }
    }
    float ss[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int c = 0; c < 2; ++c) y[e][c] = make_float2(tree_silu(y[e][c].x), tree_silu(y[e][c].y));
        const float2 sq = __ffma2_rn(y[e][0], y[e][0], __fmul2_rn(y[e][1], y[e][1]));
        ss[e] = sq.x + sq.y;
    }
    if (raw) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) ss[e] += __shfl_xor_sync(0xffffffffu, ss[e], off);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float f = scale * rsqrtf(ss[e] + eps);
            if (i0 + e < n)
                tc::st_row4(Bt, rows, row0 + i0 + e, 4 * lane, y[e][0].x * f, y[e][0].y * f, y[e][1].x * f, y[e][1].y * f);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i0 + e < n)
                *reinterpret_cast<float4*>(v + (i0 + e) * 128 + 4 * lane) = make_float4(y[e][0].x, y[e][0].y, y[e][1].x, y[e][1].y);
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
    const VtSmem lay = vt_smem(nm, gv);
    unsigned char* Bt = sm + lay.B;
    unsigned char* who = sm + lay.who;
    float* gram = reinterpret_cast<float*>(sm + lay.gram);
    float2* ent = reinterpret_cast<float2*>(sm + lay.ent);
    bf* ws = reinterpret_cast<bf*>(sm + lay.w);
    float* own = reinterpret_cast<float*>(sm + lay.own);
    int4* taps = reinterpret_cast<int4*>(sm + lay.taps);
    float* gate = reinterpret_cast<float*>(sm + lay.gate);
    float* betas = reinterpret_cast<float*>(sm + lay.beta);
    float* eg = reinterpret_cast<float*>(sm + lay.eg);
    unsigned long long* line = reinterpret_cast<unsigned long long*>(sm + lay.line);
    int* up = reinterpret_cast<int*>(sm + lay.up);
    int* off = reinterpret_cast<int*>(sm + lay.off);
    // full, freed: state atoms; done: p and r; w_ready: w and e^G r in TMEM; m_ready: M; o_done: o
    uint64_t *full = reinterpret_cast<uint64_t*>(sm + lay.bar), *freed = full + 2, *done = full + 4, *w_ready = full + 6,
             *m_ready = full + 8, *o_done = full + 10, *bar_g = full + 12;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(full + 13);
    const int tcols = nm <= 16 ? 128 : (nm <= 32 ? 256 : 512);     // products of two v-heads, then the Gram matrix
    const int halves = n > 32 ? 2 : 1, workers = 8 - 2 * halves;   // warps 0 .. workers - 1; the others make M
    if (tid == 0) {
        for (int i = 0; i < 13; ++i) mbar_init(full + i, i >= 6 && i < 8 ? 4 : (i >= 8 && i < 10 ? halves : 1));
        fence_mbar_init();
    }
    if (warp == 8) tc::alloc(tslot, tcols);
    const bf* xb = static_cast<const bf*>(J.x) + first * C;
    const bf* cb = static_cast<const bf*>(J.conv_pool) + (size_t)slot * Km1 * C;
    auto channel = [&](int what, int i) {  // first channel of k (0), q (1), v of v-head j0 + i (2)
        return (what == 0 ? Hk + h : (what == 1 ? h : 2 * Hk + j0 + i)) * D;
    };
    // the raw inputs of k and q, conv state first, into the places of M and v; those of v and z to L2
    bf* raw = reinterpret_cast<bf*>(sm + lay.M);
    for (int i = tid; i < (Km1 + n) * 32; i += kVtThreads) {
        const int row = i / 32, what = i / 16 % 2, c = i % 16 * 8;
        cp_async16(raw + row * 2 * D + what * D + c,
                   (row < Km1 ? cb + (size_t)row * C : xb + (size_t)(row - Km1) * C) + channel(what, 0) + c);
    }
    cp_async_commit();
    for (int i = tid; i < n * gv * 4; i += kVtThreads) {
        const int node = i / (4 * gv), jj = i / 4 % gv, piece = i % 4;
        tree_prefetch(piece < 2 ? xb + (size_t)node * C + channel(2, jj) + piece * 64
                                : static_cast<const bf*>(J.z) + ((size_t)(first + node) * Hv + j0 + jj) * D + (piece - 2) * 64);
    }
    // gates and parents; conv weights with the taps outside (a missing tap: 0)
    if (tid < n) {
        const int p = J.parents[first + tid];
        up[tid] = p >= 0 && p < tid ? p : -1;
    }
    for (int i = tid; i < n * gv; i += kVtThreads) {
        const int node = i / gv, jj = i % gv;
        const size_t at = (size_t)(first + node) * Hv + j0 + jj;
        gates(__bfloat162float(static_cast<const bf*>(J.a)[at]), __bfloat162float(static_cast<const bf*>(J.b)[at]),
              A.p.A_log[j0 + jj], A.p.dt_bias ? A.p.dt_bias[j0 + jj] : 0.f, false, gate[i], betas[i]);
    }
    // weights of k, q and v-heads i0, i0 + 1 (what: from .. 3), by `nt` threads
    auto stage_weights = [&](int i0, int from, int nt) {
#pragma unroll 2
        for (int k = from * D + tid; k < (2 + min(2, gv - i0)) * D; k += nt) {
            const int what = k / D;
            const bf* src = static_cast<const bf*>(A.p.conv_w) + (size_t)(channel(min(what, 2), i0 + what - 2) + k % D) * K;
            bf w4[4];
            if (K == 4) {
                *reinterpret_cast<uint2*>(w4) = __ldg(reinterpret_cast<const uint2*>(src));
            } else {
#pragma unroll
                for (int m = 0; m < 4; ++m) w4[m] = m >= 4 - K ? src[m - (4 - K)] : __float2bfloat16_rn(0.f);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) ws[(what * 4 + m) * D + k % D] = w4[m];
        }
    };
    stage_weights(0, 0, kVtThreads);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = *tslot, tgram = tm + 4 * nm;
    // the line of every node and the sum of log alpha along it, a thread per (node, v-head): two pairs a thread at most
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int k = tid + e * 256, i = k % nm, jj = k / nm;
        if (tid < 256 && i < n && jj < gv) {
            unsigned long long m = 0;
            for (int at = i; at >= 0;) {
                m |= 1ull << at;
                const int next = up[at];
                sums[e] += gate[at * gv + jj];
                at = next;
            }
            if (jj == 0) line[i] = m;
        }
    }
    if (tid >= 192 && tid - 192 < n) {  // the last tap is the node, then its ancestors, then the conv state's rows, newest first
        const int i = tid - 192;
        int at = i, row = Km1 - 1, t[4];
#pragma unroll
        for (int m = 3; m >= 0; --m) {
            const bool live = 3 - m < K;
            t[m] = !live ? i : (at >= 0 ? at : 64 + row--);
            if (live && at >= 0) at = up[at];
        }
        taps[i] = make_int4(t[0], t[1], t[2], t[3]);
    }
    cp_async_wait_all();
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // (read after the next barriers)
        const int k = tid + e * 256, i = k % nm, jj = k / nm;
        if (tid < 256 && i < n && jj < gv) {
            gate[i * gv + jj] = sums[e];
            eg[i * gv + jj] = __expf(sums[e]);
        }
    }
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {  // warp-wide; after a failure nothing waits any more
        if (ok) ok = vt_wait(bar, phase);
        return ok;
    };
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
        const uint64_t db = tc::sdesc(tc::smem_addr(Bt)), ds = tc::sdesc(tc::smem_addr(sm + lay.S)),
                       dm = tc::sdesc(tc::smem_addr(sm + lay.M));
        const uint32_t bstep = (uint32_t)(2 * nm * 128) >> 4, mstep = (uint32_t)(nm * 128) >> 4;
        const uint32_t id_n = tc::idesc_tf32(128, nm), id_2n = tc::idesc_tf32(128, 2 * nm);
        if (vt_elect()) {  // lanes are the rows of [K^; Q^] (what lies past them is never read), columns the keys
#pragma unroll 4
            for (int k = 0; k < 16; ++k)
                vt_mma(tgram, db + (k >> 2) * bstep + (k & 3) * 2, db + (k >> 2) * bstep + (k & 3) * 2, id_n, k > 0);
            tc::commit(bar_g);
        }
        __syncwarp();
        // r += w M^T of v-head i
        auto finish = [&](int i) {
            if (!wait(w_ready + (i & 1), i >> 1) || !wait(m_ready + (i & 1), i >> 1)) return;
            tc::fence_after();
            if (vt_elect()) {
                const uint32_t d = tm + (i & 1) * 2 * nm;
                for (int k = 0; k < (n + 7) / 8; ++k)
                    vt_mma_ta(d + nm, d + 8 * k, dm + ((i & 1) * ((nm + 31) / 32) + (k >> 2)) * mstep + (k & 3) * 2, id_n);
                tc::commit(o_done + (i & 1));
            }
            __syncwarp();
        };
#pragma unroll 1
        for (int a = 0; a < atoms && ok; ++a) {
            const int i = a >> 2;
            if ((a & 3) == 0 && i >= 1) finish(i - 1);
            if ((a & 3) == 0 && i >= 2 && ok) named_bar_sync(3, 160);  // o of v-head i - 2 has been read out of TMEM
            if (!wait(full + (a & 1), a >> 1)) break;
            if (vt_elect()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    vt_mma(tm + (i & 1) * 2 * nm, ds + (uint32_t)(((a & 1) * kVtAtom) >> 4) + k * 2,
                           db + (a & 3) * bstep + k * 2, id_2n, (a & 3) > 0 || k > 0);
                tc::commit(freed + (a & 1));
                if ((a & 3) == 3) tc::commit(done + (i & 1));
            }
            __syncwarp();
            if (a + 2 < atoms) {
                if (!wait(freed + (a & 1), a >> 1)) break;
                if (lane == 0) load(a + 2);
                __syncwarp();
            }
        }
        if (ok) finish(gv - 1);
        if (!ok) {  // let the copies in flight land (bounded again); the others' waits give up by themselves
            for (int i = 0; i < 2; ++i) mbar_wait(full + i, 0);
            if (lane == 0) report_device_status(kDevWaitTimeout);
        }
    } else {
        float* v = reinterpret_cast<float*>(sm + lay.v);
        const int batches = (n + 3) / 4;  // of 4 nodes
        auto conv = [&](int what, int i, int batch) {  // what: k (0) and q (1) from shared memory, v of v-head j0 + i (2)
            const int ch = channel(what, i) + 4 * lane;
            vt_conv(what < 2 ? smem_u32(raw + what * D + 4 * lane) : 0u, reinterpret_cast<const unsigned char*>(xb + ch),
                    reinterpret_cast<const unsigned char*>(cb + ch), (uint32_t)C * 2u, taps,
                    reinterpret_cast<const uint2*>(ws + (what + (i & 1)) * 4 * D),
                    A.p.conv_b ? static_cast<const bf*>(A.p.conv_b) + ch : nullptr, K, 4 * batch, n, v, Bt, 2 * nm,
                    what == 1 ? nm : 0, what == 0 ? 1.f : g.q_scale, g.l2_eps);
        };
        if (warp == 7) {  // entries before each node: scan of the numbers of proper ancestors, rounded up to pairs
            int base = 0;
            for (int i0 = 0; i0 < nm; i0 += 32) {
                const int i = i0 + lane;
                int c = i < n ? __popcll(line[i]) & ~1 : 0;
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, c, s);
                    if (lane >= s) c += x;
                }
                if (i < nm) off[i + 1] = base + c;
                base += __shfl_sync(0xffffffffu, c, 31);
            }
            if (lane == 0) off[0] = 0;
        }
#pragma unroll 1
        for (int k = warp; k < 2 * batches; k += 8) conv(k & 1, 0, k >> 1);
        fence_proxy_async_smem();
        named_bar_sync(2, kVtThreads);
#pragma unroll 1
        for (int i0 = 0; i0 < gv; i0 += 2) {  // v-heads i0 and i0 + 1
            const int two = min(2, gv - i0);
            if (i0 > 0) {
                named_bar_sync(1, 256);  // T and the first two v-heads' weights are no longer read
                stage_weights(i0, 2, 256);
            }
            if (warp < 4 && 32 * warp < 2 * nm) {  // the Gram matrix into shared memory
                if (wait(bar_g, 0)) {
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
            named_bar_sync(1, 256);
            // coefficients of the nodes' proper ancestors, a warp per node, a lane per ancestor
#pragma unroll 1
            for (int node = warp; node < n; node += 8) {
                const unsigned long long m = line[node] & ~(1ull << node);
                const float *gk = gram + node * (nm + 1), *gq = gram + (nm + node) * (nm + 1);
                const int start = off[node], c = __popcll(m);
                for (int a = lane; a < node; a += 32) {
                    if ((m >> a) & 1ull) {
                        const int at = start + __popcll(m & ((1ull << a) - 1ull));
                        const float k1 = gk[a], q1 = gq[a];
                        for (int e = 0; e < two; ++e) {
                            const float f = __expf(gate[node * gv + i0 + e] - gate[a * gv + i0 + e]);
                            ent[e * vt_entries(nm) + at] = make_float2(betas[node * gv + i0 + e] * f * k1, f * q1);
                        }
                        who[at] = (unsigned char)a;
                    }
                }
                if (lane < two && (c & 1)) ent[lane * vt_entries(nm) + start + c] = make_float2(0.f, 0.f);
                if (lane == 31) {
                    if (c & 1) who[start + c] = (unsigned char)(__ffsll((long long)m) - 1);  // (0 times the first one's row)
                    own[node] = gq[node];
                }
            }
            named_bar_sync(1, 256);
            if (warp >= workers) {
                // ---- M: column 32 half + lane of v-head i0 + e; T in the Gram matrix's place -----------
                const int e = (warp - workers) / halves, half = (warp - workers) % halves;
                if (e < two) {
                    float* T = gram + (e * ((nm + 31) / 32) + half) * nm * 32 + lane;
                    unsigned char* Mt = sm + lay.M + (e * ((nm + 31) / 32) + half) * nm * 128;
                    const float2* from = ent + e * vt_entries(nm);
                    // the entries of all nodes lie end to end: those of the next step are loaded before this step's
                    // rows of T (up to 4 entries past the last one are read, inside the layout, and not used)
                    int at = 0, end = off[1];
                    float mine = own[0];
                    float4 k01, k23;
                    uint32_t w;
                    auto fetch = [&]() {
                        k01 = *reinterpret_cast<const float4*>(from + at);
                        k23 = *reinterpret_cast<const float4*>(from + at + 2);
                        w = *reinterpret_cast<const uint16_t*>(who + at) | (uint32_t)*reinterpret_cast<const uint16_t*>(who + at + 2) << 16;
                    };
                    fetch();
#pragma unroll 1
                    for (int node = 0; node < n; ++node) {
                        const int next_end = off[min(node + 2, n)];
                        const float next_mine = own[min(node + 1, n - 1)];
                        float su[4] = {}, so[4] = {};
#pragma unroll 1
                        while (at < end) {
                            const bool four = at + 2 < end;
                            const float t0 = T[(w & 255) * 32], t1 = T[((w >> 8) & 255) * 32];
                            const float t2 = four ? T[((w >> 16) & 255) * 32] : 0.f, t3 = four ? T[(w >> 24) * 32] : 0.f;
                            const float4 a = k01, c = four ? k23 : make_float4(0.f, 0.f, 0.f, 0.f);
                            at += four ? 4 : 2;
                            fetch();
                            su[0] = fmaf(a.x, t0, su[0]);
                            so[0] = fmaf(a.y, t0, so[0]);
                            su[1] = fmaf(a.z, t1, su[1]);
                            so[1] = fmaf(a.w, t1, so[1]);
                            su[2] = fmaf(c.x, t2, su[2]);
                            so[2] = fmaf(c.y, t2, so[2]);
                            su[3] = fmaf(c.z, t3, su[3]);
                            so[3] = fmaf(c.w, t3, so[3]);
                        }
                        const float t = (node == 32 * half + lane ? 1.f : 0.f) - ((su[0] + su[1]) + (su[2] + su[3]));
                        T[node * 32] = t;
                        tc::st_elem(Mt, nm, node, lane, fmaf(mine, t, (so[0] + so[1]) + (so[2] + so[3])));
                        end = next_end;
                        mine = next_mine;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(m_ready + e);
                }
                continue;
            }
            for (int i = i0; i < i0 + two; ++i) {
#pragma unroll 1
                for (int k = warp; k < batches; k += workers) conv(2, i, k);
                uint2 zr[4];  // of the nodes below, four at a time
                auto load_z = [&](int from) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        zr[q] = __ldg(reinterpret_cast<const uint2*>(static_cast<const bf*>(J.z) +
                                                                    ((size_t)(first + min(from + workers * q, n - 1)) * Hv + j0 + i) * D) + lane);
                };
                if (warp >= 4) load_z(warp);
                named_bar_sync(4, 32 * workers);
                if (warp < 4) {
                    // ---- thread = state row: w and e^G r, then o in v's place (its own column) ------------
                    float* u = v + 32 * warp + lane;
                    const uint32_t tr = tc::taddr(tm, 32 * warp, (i & 1) * 2 * nm);
                    unsigned long long bad = 0ull;  // nodes whose w is an infinity or NaN here
                    wait(done + (i & 1), i >> 1);
                    tc::fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < n; c0 += 8) {
                        uint32_t rk[8], rq[8];
                        vt_ld8(tr + c0, rk);
                        vt_ld8(tr + nm + c0, rq);
                        float be[8], e[8], vi[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const int node = min(c0 + c, n - 1);
                            be[c] = betas[node * gv + i];
                            e[c] = eg[node * gv + i];
                            vi[c] = u[node * D];
                        }
                        tc::ld_wait();
                        float wv[8], ro[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float w = be[c] * (vi[c] - e[c] * __uint_as_float(rk[c]));
                            ro[c] = e[c] * __uint_as_float(rq[c]);
                            // M is 0 off the line, but 0 times an infinity or NaN is not: those are added below
                            const bool fine = isfinite(w) && c0 + c < n;
                            wv[c] = fine ? tc::to_tf32_rn(w) : 0.f;
                            if (!fine && c0 + c < n) {
                                bad |= 1ull << (c0 + c);
                                u[(c0 + c) * D] = w;
                            }
                        }
                        vt_st8(tr + c0, wv);
                        vt_st8(tr + nm + c0, ro);
                    }
                    tc::st_wait();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(w_ready + (i & 1));
                    load_z(warp);
                    wait(o_done + (i & 1), i >> 1);
                    tc::fence_after();
                    const unsigned char* Mt = sm + lay.M + (i & 1) * ((nm + 31) / 32) * nm * 128;
#pragma unroll 1
                    for (int c0 = (n - 1) & ~7; c0 >= 0; c0 -= 8) {  // from the last node on: see below
                        uint32_t ro[8];
                        vt_ld8(tr + nm + c0, ro);
                        tc::ld_wait();
                        if (bad) {
                            // a line's nodes come before its end, so their w are still there
                            for (int node = min(c0 + 7, n - 1); node >= c0; --node) {
                                float more = 0.f;
                                for (unsigned long long m = bad & line[node]; m; m &= m - 1) {
                                    const int a = __ffsll((long long)m) - 1;
                                    more = fmaf(*reinterpret_cast<const float*>(Mt + tc::sw_off(nm, node, a)), u[a * D], more);
                                }
                                float o = 0.f;
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    if (c0 + c == node) o = __uint_as_float(ro[c]);
                                u[node * D] = o + more;
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                if (c0 + c < n) u[(c0 + c) * D] = __uint_as_float(ro[c]);
                        }
                        __syncwarp();
                    }
                    tc::fence_before();
                }
                named_bar_sync(4, 32 * workers);
                if (warp < 4 && i + 2 < gv) asm volatile("bar.arrive 3, 160;" ::: "memory");  // this v-head's columns are free
                // gated RMSNorm, a warp per node, four nodes at once, four channels to a lane
                const uint2 nw = __ldg(reinterpret_cast<const uint2*>(A.p.norm_w) + lane);
                const float2 w01 = vt_two(nw.x), w23 = vt_two(nw.y);
#pragma unroll 1
                for (int n0 = warp; n0 < n; n0 += 4 * workers) {
                    if (n0 > warp) load_z(n0);
                    float4 o[4];
                    float ss[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[q] = *reinterpret_cast<const float4*>(v + min(n0 + workers * q, n - 1) * D + 4 * lane);
                        ss[q] = fmaf(o[q].x, o[q].x, fmaf(o[q].y, o[q].y, fmaf(o[q].z, o[q].z, o[q].w * o[q].w)));
                    }
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                        for (int q = 0; q < 4; ++q) ss[q] += __shfl_xor_sync(0xffffffffu, ss[q], off);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int node = n0 + workers * q;
                        const float inv = rsqrtf(fmaf(ss[q], 1.f / D, g.norm_eps));
                        const float2 z01 = vt_two(zr[q].x), z23 = vt_two(zr[q].y);
                        const __nv_bfloat162 y01 = __floats2bfloat162_rn(o[q].x * inv * w01.x * tree_silu(z01.x),
                                                                         o[q].y * inv * w01.y * tree_silu(z01.y));
                        const __nv_bfloat162 y23 = __floats2bfloat162_rn(o[q].z * inv * w23.x * tree_silu(z23.x),
                                                                         o[q].w * inv * w23.y * tree_silu(z23.y));
                        uint2 out;
                        memcpy(&out.x, &y01, 4);
                        memcpy(&out.y, &y23, 4);
                        if (ok && node < n)
                            *(reinterpret_cast<uint2*>(static_cast<bf*>(J.y) + ((size_t)(first + node) * Hv + j0 + i) * D) + lane) = out;
                    }
                }
                if (i + 1 < gv) named_bar_sync(4, 32 * workers);  // o is read: its place takes the next v
            }
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
    VtArgs A{g, p, job, (job.max_nodes + 15) / 16 * 16, g.G};
    // few trees: a CTA per v-head; and as many v-heads as shared memory holds the decays of
    if ((long)job.B * g.Hk < sm_count()) A.gv = 1;
    while (vt_smem(A.nm, A.gv).total + 1024 > 227 * 1024 || A.g.G % A.gv) --A.gv;
    return launch_pdl(k_tree_verify_tc, dim3((unsigned)(g.Hv / A.gv), (unsigned)job.B), dim3(kVtThreads),
                      (size_t)vt_smem(A.nm, A.gv).total + 1024, st, map, A);
}

// ---- commit ---------------------------------------------------------------------
// One CTA per (v-head, sequence), a cluster per k-head.  A warp holds D / 8 state rows in registers
// through all rows of the path (a state row's update touches no other row), 8 lanes to a row as in
// k_tree_verify, so the state is read once and written once, and shared memory holds only
// the inputs, k and v of a chunk of path rows at a time.  HBM-bound: while a CTA prepares k and v, its state is on the
// way to L2, asked for by the CTA that ran a wave before it.  The G CTAs of a k-head read the same conv rows of k,
// which one of them replaces: the cluster barrier stands between.
template <typename TA>
constexpr int kComChunk = sizeof(TA) == 2 ? 16 : 8;

struct CommitArgs {
    Geom g;
    LayerParams p;
    TreeCommitJob job;
    int ahead;  // sequences between a CTA and the one whose state it asks for
};

template <int D, typename TA>
__global__ void __launch_bounds__(kTreeThreads, 2) k_tree_commit(const __grid_constant__ CommitArgs A) {
    using L = Act<TA>;
    constexpr int LPN = D / 4, NPW = 32 / LPN;  // lanes of a path row's channels, rows of a warp (conv)
    constexpr int RL = D / 32;                  // state rows and 4-column chunks of a lane
    constexpr int nwarp = kTreeThreads / 32, kComRows = kComChunk<TA>;
    const Geom& g = A.g;
    const TreeCommitJob& J = A.job;
    const int gi = blockIdx.x, h = blockIdx.y, j = h * g.G + gi, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hk = g.Hk, Hv = g.Hv, K = g.K, Km1 = g.K - 1, C = g.C_ch;
    const bool raw = g.flags & kFlagRawQKV;
    __shared__ __align__(16) float ks[kComRows][D], vs[kComRows][D];
    __shared__ __align__(16) TA ws[2][5][D];                // conv taps and bias of k and v
    __shared__ __align__(16) TA hs[kComRows + 3][3][D];     // raw inputs of q, k, v: K - 1 before the chunk, then its rows
    __shared__ float alpha_s[kTreeMax], beta_s[kTreeMax];
    __shared__ int rows[kTreeMax];
    __shared__ int n_s;
    griddep_wait();
    griddep_launch_dependents();
    const int slot = J.slot_idx[b];
    const int64_t first = J.cu_rows[b], count = (int64_t)J.cu_rows[b + 1] - first;
    for (int far = b < A.ahead ? 0 : A.ahead; far <= A.ahead; far += A.ahead) {  // (the first wave asks for its own too)
        if (b + far >= J.B) break;
        const int s2 = J.slot_idx[b + far];
        if (s2 >= 0 && s2 < J.n_slots && J.cu_rows[b + far + 1] > J.cu_rows[b + far]) {
            const float* p = J.state_pool + ((size_t)s2 * Hv + j) * D * D;
            for (int i = tid; i < D * D / 32; i += kTreeThreads) tree_prefetch(p + i * 32);
        }
    }
    if (slot < 0 || slot >= J.n_slots || first < 0 || count < 1 || count > J.max_rows || first + count > J.n_rows)
        return;  // the whole cluster shares b
    const int l8 = lane & 7, grp = lane >> 3, row0 = warp * (D / 8) + grp;  // state row r * 4 + group, columns 4 l8 + 32 c
    float* Sg = J.state_pool + (((size_t)slot * Hv + j) * D + row0) * D + 4 * l8;
    float4 S[RL][RL];
#pragma unroll
    for (int r = 0; r < RL; ++r)
#pragma unroll
        for (int c = 0; c < RL; ++c) S[r][c] = *reinterpret_cast<const float4*>(Sg + (size_t)r * 4 * D + 32 * c);
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
    auto channel = [&](int kind) { return (kind == 0 ? h : (kind == 1 ? Hk + h : 2 * Hk + j)) * D; };  // q, k, v
    if (!raw) {
        for (int i = tid; i < 2 * D; i += kTreeThreads) {
            const int ch = channel(1 + i / D) + i % D;
            TA zero;
            L::st(&zero, 0, 0.f);
#pragma unroll
            for (int t = 0; t < 4; ++t) {  // (taps are aligned at the newest)
                const int m = t - (4 - K);
                ws[i / D][t][i % D] = m >= 0 ? static_cast<const TA*>(A.p.conv_w)[(size_t)ch * K + m] : zero;
            }
            ws[i / D][4][i % D] = A.p.conv_b ? static_cast<const TA*>(A.p.conv_b)[ch] : zero;
        }
    }
    __syncthreads();
    const int n = n_s;
    if (n == 0) return;  // no row that exists (the whole cluster)
    const TA* x = static_cast<const TA*>(J.x);
    TA* cp = static_cast<TA*>(J.conv_pool) + (size_t)slot * Km1 * C;
    for (int t0 = 0; t0 < n; t0 += kComRows) {
        const int m = min(kComRows, n - t0);
        // the chunk's raw inputs, all on their way at once (through shared memory: the state has the registers): input p
        // of the sequence is row p of the conv state, then the path's rows
        {
            constexpr int PER = D * (int)sizeof(TA) / 16;  // 16-byte pieces of a row's head
            for (int i = tid; i < (m + Km1) * 3 * PER; i += kTreeThreads) {
                const int row = i / (3 * PER), kind = i / PER % 3, c = i % PER * (16 / (int)sizeof(TA)), p = t0 + row;
                cp_async16(&hs[row][kind][c], (p < Km1 ? cp + (size_t)p * C : x + (size_t)rows[p - Km1] * C) + channel(kind) + c);
            }
            cp_async_commit();
        }
        if (t0 == 0) {
            const bool direct = g.flags & kFlagGatesDirect;
            for (int t = tid - (kTreeThreads - 64); t >= 0 && t < n; t += 64) {
                float gl, beta;
                gates(L::ld(J.a, (size_t)rows[t] * Hv + j), L::ld(J.b, (size_t)rows[t] * Hv + j), direct ? 0.f : A.p.A_log[j],
                      !direct && A.p.dt_bias ? A.p.dt_bias[j] : 0.f, direct, gl, beta);
                alpha_s[t] = expf(gl);
                beta_s[t] = beta;
            }
        }
        cp_async_wait_all();
        __syncthreads();
        // the conv state is read (rows past the first K - 1 do not reach it): the cluster's other CTAs may replace it
        if (t0 == 0) cluster_arrive_release();
        // conv + SiLU of k and v, L2 norm of k: an LPN-lane group has a path row's D channels
        {
            const int sub = lane / LPN, c4 = (lane % LPN) * 4;
            auto ld4 = [&](const TA* p) { return make_float4(L::ld(p, 0), L::ld(p, 1), L::ld(p, 2), L::ld(p, 3)); };
#pragma unroll 2
            for (int unit = warp; unit < 2 * ((m + NPW - 1) / NPW); unit += nwarp) {
                const int kind = unit & 1, i0 = (unit >> 1) * NPW + sub, i = min(i0, m - 1);
                float4 y = ld4(&hs[i + Km1][1 + kind][c4]);
                if (!raw) {
                    const float4 v3 = y;
                    y = ld4(&ws[kind][4][c4]);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        if (t < 4 - K) continue;
                        const float4 w = ld4(&ws[kind][t][c4]), v = t == 3 ? v3 : ld4(&hs[i + Km1 - 3 + t][1 + kind][c4]);
                        y.x = fmaf(w.x, v.x, y.x);
                        y.y = fmaf(w.y, v.y, y.y);
                        y.z = fmaf(w.z, v.z, y.z);
                        y.w = fmaf(w.w, v.w, y.w);
                    }
                    y = make_float4(tree_silu(y.x), tree_silu(y.y), tree_silu(y.z), tree_silu(y.w));
                }
                if (kind == 0 && !(g.flags & kFlagNoL2)) {
                    float ss = fmaf(y.x, y.x, fmaf(y.y, y.y, fmaf(y.z, y.z, y.w * y.w)));
#pragma unroll
                    for (int o = LPN / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float f = rsqrtf(ss + g.l2_eps);
                    y = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
                }
                if (i0 < m) *reinterpret_cast<float4*>(&(kind == 0 ? ks : vs)[i0][c4]) = y;
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int t = 0; t < m; ++t) {
            float4 k[RL];
            float2 d[RL];
            float dot[RL];
#pragma unroll
            for (int c = 0; c < RL; ++c) k[c] = *reinterpret_cast<const float4*>(&ks[t][4 * l8 + 32 * c]);
#pragma unroll
            for (int r = 0; r < RL; ++r) {
                d[r] = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < RL; ++c) d[r] = tree_dot(S[r][c], k[c], d[r]);
                dot[r] = d[r].x + d[r].y;
            }
            // lane l8 of a group: the sum of state row l8 / (8 / RL); beta (v - alpha S k) of it, handed to the group
            const float sum = tree_sum8<RL>(dot, lane);
            const float alpha = alpha_s[t0 + t];
            const float be = beta_s[t0 + t] * (vs[t][row0 + (l8 / (8 / RL)) * 4] - alpha * sum);
            const float2 al2 = make_float2(alpha, alpha);
#pragma unroll
            for (int r = 0; r < RL; ++r) {
                const float ber = __shfl_sync(0xffffffffu, be, (lane & 24) + r * (8 / RL));
                const float2 b2 = make_float2(ber, ber);
#pragma unroll
                for (int c = 0; c < RL; ++c) {
                    const float2 lo = __ffma2_rn(al2, make_float2(S[r][c].x, S[r][c].y), __fmul2_rn(b2, make_float2(k[c].x, k[c].y)));
                    const float2 hi = __ffma2_rn(al2, make_float2(S[r][c].z, S[r][c].w), __fmul2_rn(b2, make_float2(k[c].z, k[c].w)));
                    S[r][c] = make_float4(lo.x, lo.y, hi.x, hi.y);
                }
            }
        }
        if (t0 + kComRows < n) __syncthreads();  // ks, vs and the inputs are read
    }
    // the new conv state: the last K - 1 raw inputs, bit for bit, from shared memory
#pragma unroll
    for (int r = 0; r < RL; ++r)
#pragma unroll
        for (int c = 0; c < RL; ++c) *reinterpret_cast<float4*>(Sg + (size_t)r * 4 * D + 32 * c) = S[r][c];
    cluster_wait_acquire();
    const int tail = (n - 1) % kComRows + 1;  // rows of the last chunk
    for (int c = tid; c < 3 * D; c += kTreeThreads) {
        const int kind = c / D;
        if (kind < 2 && c % g.G != gi) continue;  // (q and k channels: one CTA of the cluster each)
        for (int m = 0; m < Km1; ++m) cp[(size_t)m * C + channel(kind) + c % D] = hs[tail + m][kind][c % D];
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
    const CommitArgs A{g, p, job, std::max(1, 2 * sm_count() / g.Hv)};
    GDN_BY_TYPE(launch_commit_t);
}

cudaError_t take_device_status_tree(unsigned* out) { return take_device_status_tu(out); }

}  // namespace gdn
