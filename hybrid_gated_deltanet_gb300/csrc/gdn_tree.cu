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
// once for all nodes, no state of a node is formed, and no exponent is positive.  This is the
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
__device__ __forceinline__ float tree_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// x sigmoid(x) by the SFU's exponential and reciprocal, five instructions (the functions of the math library spend as many
// again on subnormal arguments, which the sum with 1 absorbs here): 2^-21 relative at the sizes of a conv's outputs
__device__ __forceinline__ float tree_silu(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + tree_ex2(x * -1.4426950408889634f)));
    return x * r;
}

// The sum of log alpha along a line, as a pair of floats s + lo: lo takes what the rounding of s leaves out.  The decay between a
// node and an ancestor is the exponential of the difference of two such sums, and after strong decays a single float would have
// few digits left for the weak ones that follow (eight nodes of -128, then gates of -0.005: 1e-4 of the decay).
__device__ __forceinline__ void tree_add(float& s, float& lo, float x) {
    const float t = s + x, b = t - s;
    lo += (s - (t - b)) + (x - b);
    s = t;
}
// A gate as a term of these sums.  An alpha of e^-1000 is 0 in fp32, as one of e^-inf is, and so is every decay across it; but the
// sums stay finite, and nodes below it differ by what comes after it
constexpr float kTreeErased = -1000.f;
__device__ __forceinline__ float tree_gate(float g) { return g < kTreeErased ? kTreeErased : g; }  // (NaN stays)

// entries of a tree's nodes: a node's proper ancestors, rounded up to groups of 4
__host__ __device__ inline int tree_entries(int n) { return n * (n - 1) / 2 + 3 * n; }

struct TreeSmem {
    int k, q, u, p, r, w, ent, node, lo, anc, up, off, taps, total;
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
    s.lo = o; o = (o + n * 4 + 7) & ~7;           // G's lower part
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
// node against 4 d^2 bytes of state per tree, and as much again for the shuffles, the conv and the line sums (8 chains of
// 20 nodes, 48 v-heads, d = 128, fp32: 32 us, 14 us per CTA in one wave and a quarter).
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
    float* lo = reinterpret_cast<float*>(smem + lay.lo);
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
        nd[tid] = make_float4(beta, tree_gate(gl), 0.f, 0.f);
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
    float G = 0.f, Glo = 0.f;
    if (tid < n) {  // the node's line, and the decay along it
        unsigned long long m = 0;
        for (int i = tid; i >= 0; i = up[i]) {
            m |= 1ull << i;
            tree_add(G, Glo, nd[i].y);
        }
        anc[tid] = m;
        lo[tid] = Glo;
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
    if (tid < n) nd[tid] = make_float4(beta, G, expf(G + Glo), 0.f);
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
                    const float f = expf((me.y - nd[a].y) + (lo[i] - lo[a]));
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
// One CTA per (k-head, tree).  With p_j = S_0 k_j, r_j = S_0 q_j and w_j = beta_j (v_j - e^{G_j} p_j), the sums above are
//   u = T w,   o_i = e^{G_i} r_i + sum_j P_ij u_j,   T = (I + A)^-1,
// with A (keys: beta_i e^{G_i - G_j} k_i . k_j, j a proper ancestor) and P (queries: e^{G_i - G_j} q_i . k_j, j = i too) of
// n x n per v-head and the same for all 128 state rows.  So (products TF32, fp32 accumulation):
//   [K^; Q^] K^T    M = 128, N = nm, once: the products of the nodes' keys and queries with keys.  These are made to 2^-20 of
//                   |q| |k| (what TF32 leaves out of the factors, times the values, is added by bf16 products): one of them may
//                   be all of a node's output, the norm divides by its size, and of a small one TF32's 2^-11 of
//                   |q| |k| would be much (y off by 20% where |q . k| is 1.5e-4 of it);
//   S_0 [K^; Q^]^T  per v-head, M = 128 state rows, N = 2 nm, S_0 as it lies in the pool (fp32, brought by tensor
//                   TMA 32 columns at a time; the tensor core reads its leading 10 fraction bits, as it does of K^ and
//                   Q^ rounded): p and r in TMEM;
//   u = w T^T       w in TMEM in p's place;
//   r += u P^T      u in TMEM, rounded by way of registers.
// T is made in place of A, in fp32, by a warp (two above 32 nodes) per v-head: blocks of 16 on the diagonal by
// substitution, a column to a lane; then T21 = -T22 A21 T11 for the blocks of 16 and of 32 below it.  TF32's 2^-11 per
// operand is a quarter of the bf16 rounding of y; the decays, T's sums and the norms are fp32.
// The phases are short, so that latency and instructions bound the kernel (64 trees of up to 32 nodes, 16 / 32 heads:
// 81 us, 2.1 TB/s of the state's bytes; HBM is a quarter busy, the issue slots 39%).  Two CTAs share an SM up to 32 nodes:
// the state's place in shared memory is half a tile for that.  Measured there, in an earlier build of 76 us: 16 warps a CTA
// 87 us, 12 warps 84, 8 warps 76 (what a warp does once weighs more than its waiting); three CTAs an SM, with one v-head at a
// time and a quarter tile, 74 us, but 83 against 78 at 16 trees of 64 nodes and 48 v-heads.
constexpr int kVtWorkers = 7;    // and a warp that drives the copies and the products
constexpr int kVtThreads = 32 * (kVtWorkers + 1);
constexpr int kVtNorm = 2;       // nodes that a warp takes at a time in the norm
constexpr int kVtRows = 4;       // warps 0 .. 3 have the state rows: TMEM lanes by quarter
constexpr int kVtAtom = 16384;   // 128 state rows x 32 columns

struct VtSmem {
    int S, B, L, A, P, v, w, taps, gate, lo, beta, eg, line, up, bad, bar, total;
};

// atoms of the ring that are free from the start: L has the others' place until the Gram product is done
__host__ __device__ inline int vt_early(int nm, int apart) { return apart || nm > 32 ? 2 : (nm > 16 ? 0 : 1); }

__host__ __device__ inline VtSmem vt_smem(int nm, int gv, int apart) {  // nm: nodes, rounded up to 16; apart: L has a place of its own
    const int two = gv > 1 ? 2 : 1;  // v-heads are taken two at a time
    VtSmem s;
    int o = 0;
    s.S = o; o += 2 * kVtAtom;                       // ring of state atoms
    s.B = o; o += 2 * nm * 512;                      // [K^; Q^]: 4 atoms of 2 nm rows x 128 bytes
    s.A = o; o += two * ((nm + 31) / 32) * nm * 128; // A, then T, of two v-heads: atoms of nm rows x 32 columns
    s.P = o; o += two * ((nm + 31) / 32) * nm * 128; // (at first, from A on: raw q and k of [K - 1 + n] rows)
    s.v = o; o += nm * 512;                          // v, then o: [node][row]
    // what rounding [K^; Q^] left out and [K^; Q^] itself, in bf16 (2 + 2 atoms of 2 nm rows x 64 columns), until the Gram product
    // has them: in the ring, or behind the raw q and k
    s.L = apart ? o : (nm <= 32 ? s.S + vt_early(nm, 0) * kVtAtom : ((s.A + (nm + 3) * 512 + 1023) & ~1023));
    if ((apart || nm > 32) && o < s.L + 2 * nm * 512) o = s.L + 2 * nm * 512;
    s.w = o; o += (2 + two) * 4 * 128 * 2;           // conv weights of k, q and two v-heads: [4 taps][128]
    s.taps = o; o += nm * 16;                        // rows of the conv taps: K - 1 rows of the conv state, then the nodes
    s.gate = o; o += nm * gv * 4;                    // [v-head][node]: log2 alpha, then its sum G along the line
    s.lo = o; o += nm * gv * 4;                      // G's lower part
    s.beta = o; o += nm * gv * 4;
    s.eg = o; o += nm * gv * 4;                      // 2^G
    s.line = o; o += nm * 8;
    s.up = o; o += nm * 4;
    s.bad = o; o += 5 * 8;                           // nodes with an infinite or NaN w, and u, per v-head of the pair; and
                                                     // whether A or P has one
    s.bar = o; o += 20 * 8;
    // the Gram product reads 128 rows of each atom of B and L, whatever 2 nm is: all of them lie inside the allocation
    const int end = (s.L > s.B ? s.L : s.B) + 3 * 2 * nm * 128 + kVtAtom;
    s.total = o > end ? o : end;
    return s;
}

struct VtArgs {
    Geom g;
    LayerParams p;
    TreeJob job;
    int nm, gv;  // gv: v-heads per CTA (G, or 1 where that fills the card better)
    int apart;   // L has a place of its own
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
__device__ __forceinline__ void vt_mma_ta(uint32_t d, uint32_t a, uint64_t bd, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(bd), "r"(idesc), "r"(acc)
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

// the convolution and SiLU of the warp's 128 channels (4 to a lane) at NODES nodes: u: inputs by tap, w: [tap][128] weights
template <int NODES>
__device__ __forceinline__ void vt_taps(const uint2 (&u)[NODES][4], const uint2* w, const __nv_bfloat16* bias, int K,
                                        float2 (&y)[NODES][2]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < NODES; ++e)
#pragma unroll
        for (int c = 0; c < 2; ++c)  // (a bias may start at any element: no wider loads)
            y[e][c] = bias ? make_float2(__bfloat162float(bias[2 * c]), __bfloat162float(bias[2 * c + 1])) : make_float2(0.f, 0.f);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if (m < 4 - K) continue;  // a tap that d_conv < 4 does not have
        const uint2 wm = w[m * 32 + lane];
        const float2 w01 = vt_two(wm.x), w23 = vt_two(wm.y);
#pragma unroll
        for (int e = 0; e < NODES; ++e) {
            y[e][0] = __ffma2_rn(w01, vt_two(u[e][m].x), y[e][0]);
            y[e][1] = __ffma2_rn(w23, vt_two(u[e][m].y), y[e][1]);
        }
    }
#pragma unroll
    for (int e = 0; e < NODES; ++e)
#pragma unroll
        for (int c = 0; c < 2; ++c) y[e][c] = make_float2(tree_silu(y[e][c].x), tree_silu(y[e][c].y));
}

// Both functions: one copy of the code serves every call (the phases run once per CTA, and copies in line were bound by
// instruction fetch), and all loads of a call are on their way at once.

// v at the nodes i0 .. i0 + NODES - 1, inputs in global memory (x: from K - 1 rows before the first node's), to
// v[node][4 lane]
template <int NODES>
__device__ __noinline__ void vt_conv_v(const unsigned char* x, const unsigned char* state, uint32_t row_bytes, const int4* taps,
                                       const uint2* w, const __nv_bfloat16* bias, int K, int i0, int n, float* v) {
    uint2 u[NODES][4];
#pragma unroll
    for (int e = 0; e < NODES; ++e) {
        const int4 t4 = taps[min(i0 + e, n - 1)];
        const int tap[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
        for (int m = 0; m < 4; ++m)
            u[e][m] = __ldg(reinterpret_cast<const uint2*>((tap[m] < K - 1 ? state : x) + (uint64_t)(uint32_t)tap[m] * row_bytes));
    }
    float2 y[NODES][2];
    vt_taps<NODES>(u, w, bias, K, y);
#pragma unroll
    for (int e = 0; e < NODES; ++e)
        if (i0 + e < n)
            *reinterpret_cast<float4*>(v + (i0 + e) * 128 + 4 * (threadIdx.x & 31)) =
                make_float4(y[e][0].x, y[e][0].y, y[e][1].x, y[e][1].y);
}

// Four values to row r of the operands: rounded to TF32 to `tile`, and to `low` in bf16, atoms of 64 columns, what that rounding
// left out (the first two atoms) and the value (the other two)
__device__ __forceinline__ void vt_split4(unsigned char* tile, unsigned char* low, int rows, int r, int k, const float (&x)[4]) {
    float h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = tc::to_tf32_rn(x[e]);
    *reinterpret_cast<float4*>(tile + tc::sw_off(rows, r, k)) = make_float4(h[0], h[1], h[2], h[3]);
    const __nv_bfloat162 pair[4] = {__floats2bfloat162_rn(x[0] - h[0], x[1] - h[1]), __floats2bfloat162_rn(x[2] - h[2], x[3] - h[3]),
                                    __floats2bfloat162_rn(x[0], x[1]), __floats2bfloat162_rn(x[2], x[3])};
    uint2 u[2];
    memcpy(u, pair, sizeof u);
    unsigned char* to = low + (k >> 6) * rows * 128 + tc::h_off(r, (k >> 3) & 7) + (k & 4) * 2;
    *reinterpret_cast<uint2*>(to) = u[0];
    *reinterpret_cast<uint2*>(to + 2 * rows * 128) = u[1];
}

// k, then q, at the same nodes: inputs in shared memory from `raw` on (conv state first; a row is k's 256 bytes, then
// q's), L2-normalised to rows `node` and nm + node of [K^; Q^], q times `scale` too
template <int NODES>
__device__ __noinline__ void vt_conv_kq(uint32_t raw, const int4* taps, const uint2* w, const __nv_bfloat16* bias_k,
                                        const __nv_bfloat16* bias_q, int K, int i0, int n, unsigned char* Bt, unsigned char* Lt, int nm,
                                        float scale, float eps) {
    const int lane = threadIdx.x & 31;
    float2 k[NODES][2], y[NODES][2];
    float kk[NODES], qq[NODES];
#pragma unroll 1
    for (int what = 0; what < 2; ++what) {
        uint2 u[NODES][4];
#pragma unroll
        for (int e = 0; e < NODES; ++e) {
            const int4 t4 = taps[min(i0 + e, n - 1)];
            const int tap[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
            for (int m = 0; m < 4; ++m)
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                             : "=r"(u[e][m].x), "=r"(u[e][m].y)
                             : "r"(raw + what * 256 + tap[m] * 512));
        }
        vt_taps<NODES>(u, w + what * 128, what ? bias_q : bias_k, K, y);
        if (what == 0) {
#pragma unroll
            for (int e = 0; e < NODES; ++e)
#pragma unroll
                for (int c = 0; c < 2; ++c) k[e][c] = y[e][c];
        }
    }
#pragma unroll
    for (int e = 0; e < NODES; ++e) {
        const float2 a = __ffma2_rn(k[e][0], k[e][0], __fmul2_rn(k[e][1], k[e][1]));
        const float2 b = __ffma2_rn(y[e][0], y[e][0], __fmul2_rn(y[e][1], y[e][1]));
        kk[e] = a.x + a.y;
        qq[e] = b.x + b.y;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int e = 0; e < NODES; ++e) {
            kk[e] += __shfl_xor_sync(0xffffffffu, kk[e], off);
            qq[e] += __shfl_xor_sync(0xffffffffu, qq[e], off);
        }
#pragma unroll
    for (int e = 0; e < NODES; ++e) {
        if (i0 + e >= n) continue;
        const float fk = rsqrtf(kk[e] + eps), fq = scale * rsqrtf(qq[e] + eps);
        const float kv[4] = {k[e][0].x * fk, k[e][0].y * fk, k[e][1].x * fk, k[e][1].y * fk};
        const float qv[4] = {y[e][0].x * fq, y[e][0].y * fq, y[e][1].x * fq, y[e][1].y * fq};
        vt_split4(Bt, Lt, 2 * nm, i0 + e, 4 * lane, kv);
        vt_split4(Bt, Lt, 2 * nm, nm + i0 + e, 4 * lane, qv);
    }
}

// A, T and P: [atom of 32 columns][rows][128 bytes], swizzled
__device__ __forceinline__ float* vt_at(unsigned char* t, int rows, int r, int c) {
    return reinterpret_cast<float*>(t + tc::sw_off(rows, r, c));
}

__device__ __forceinline__ float4 vt_ld4(uint32_t at) {
    float4 x;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ float vt_ld1(uint32_t at) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ void vt_st1(uint32_t at, float x) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory"); }

// the inverses of I + A's blocks of 16 on the diagonal at rows 16 b0 and, by the upper half of the warp, 16 (b0 + 1):
// lane = column, its values in registers
__device__ __noinline__ void vt_diag(unsigned char* A, int rows, int b0, int nb) {
    const int lane = threadIdx.x & 31, c = lane & 15;
    const bool on = b0 + (lane >> 4) < nb;
    const int r0 = 16 * (on ? b0 + (lane >> 4) : b0);
    const uint32_t at = smem_u32(vt_at(A, rows, r0, r0)), col = at + (c & 3) * 4;  // (rows r0 + i: i & 7 picks the swizzle)
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < i; j += 4) {
            const float4 a = vt_ld4((at ^ (uint32_t)(((j >> 2) ^ (i & 7)) << 4)) + i * 128);
            s[0] = fmaf(a.x, t[j], s[0]);
            if (j + 1 < i) s[1] = fmaf(a.y, t[j + 1], s[1]);
            if (j + 2 < i) s[0] = fmaf(a.z, t[j + 2], s[0]);
            if (j + 3 < i) s[1] = fmaf(a.w, t[j + 3], s[1]);
        }
        t[i] = (c == i ? 1.f : 0.f) - (s[0] + s[1]);
    }
    __syncwarp();
    if (on) {
#pragma unroll
        for (int i = 0; i < 16; ++i) vt_st1((col ^ (uint32_t)(((c >> 2) ^ (i & 7)) << 4)) + i * 128, t[i]);
    }
    __syncwarp();
}

// the two warps that make T of v-head e of the pair (constant names: a computed one takes all 16 barriers of the CTA)
__device__ __forceinline__ void vt_pair_sync(int e) {
    if (e == 0)
        named_bar_sync(5, 64);
    else
        named_bar_sync(6, 64);
}

// T in A's place over the nodes' lines alone, row by row; lane = two columns
__device__ __noinline__ void vt_lines(unsigned char* A, int rows, int n, const unsigned long long* line) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        float s[2] = {0.f, 0.f};
        for (unsigned long long m = line[i] & ~(1ull << i); m; m &= m - 1) {
            const int j = __ffsll((long long)m) - 1;
            const float a = *vt_at(A, rows, i, j);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (lane + 32 * e < rows) s[e] = fmaf(a, *vt_at(A, rows, j, lane + 32 * e), s[e]);
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (lane + 32 * e < rows) *vt_at(A, rows, i, lane + 32 * e) = (lane + 32 * e == i ? 1.f : 0.f) - s[e];
        __syncwarp();
    }
}

// T21 = -T22 (A21 T11) in A21's place: rows r0 .. r0 + k2 - 1, columns c0 .. c0 + k1 - 1 (both diagonal blocks are
// inverted).  The warp has the 16 columns from `col` on, a lane a column and 8 rows of each 16; with two warps (pair >= 0)
// the one waits for the other before A21 is overwritten.
__device__ __noinline__ void vt_below(unsigned char* A, int rows, int r0, int c0, int k1, int k2, int col, int pair) {
    const int lane = threadIdx.x & 31, c = col + (lane & 15), g = 8 * (lane >> 4);
    // (row & 7 picks the swizzle, so that with rows and columns in steps of 8 and 4 the addresses differ by constants)
    const uint32_t own = smem_u32(vt_at(A, rows, r0 + g, c));
    auto product = [&](float (&acc)[2][8], int lk, int K) {  // rows r0 + 16 p + g + e: L[.][lk + k] R[lk + k][c]
        uint32_t right = smem_u32(vt_at(A, rows, lk, c)), left = smem_u32(vt_at(A, rows, r0 + g, lk));
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[p][e] = 0.f;
#pragma unroll 1
        for (int k = 0; k < K; k += 8) {
#pragma unroll
            for (int h = 0; h < 8; h += 4) {
                float x[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) x[q] = vt_ld1((right ^ (uint32_t)((h + q) << 4)) + (h + q) * 128);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    if (16 * p >= k2) break;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 l = vt_ld4((left ^ (uint32_t)(((h >> 2) ^ e) << 4)) + (16 * p + e) * 128);
                        acc[p][e] = fmaf(l.x, x[0], fmaf(l.y, x[1], fmaf(l.z, x[2], fmaf(l.w, x[3], acc[p][e]))));
                    }
                }
            }
            right += 8 * 128;
            left ^= (uint32_t)(((k >> 2) ^ ((k + 8) >> 2)) << 4);  // the next 8 columns (K <= 32: inside the atom)
        }
    };
    auto store = [&](const float (&acc)[2][8], float sign) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (16 * p >= k2) break;
#pragma unroll
            for (int e = 0; e < 8; ++e) vt_st1((own ^ (uint32_t)(e << 4)) + (16 * p + e) * 128, sign * acc[p][e]);
        }
    };
    float acc[2][8];
    product(acc, c0, k1);
    if (pair >= 0)
        vt_pair_sync(pair);
    else
        __syncwarp();
    store(acc, 1.f);
    __syncwarp();
    product(acc, r0, k2);
    __syncwarp();
    store(acc, -1.f);
    __syncwarp();
}

// CTAS: what registers allow for on an SM
template <int CTAS>
__global__ void __launch_bounds__(kVtThreads, CTAS)
    k_tree_verify_tc(const __grid_constant__ CUtensorMap ts, const __grid_constant__ VtArgs A) {
    constexpr int D = 128, NODES = CTAS == 3 ? 2 : 3;  // nodes that a warp takes at a time in the conv
    using bf = __nv_bfloat16;
    const Geom& g = A.g;
    const TreeJob& J = A.job;
    const int nm = A.nm, gv = A.gv, per_k = g.G / gv;
    const int h = blockIdx.x / per_k, j0 = h * g.G + (blockIdx.x % per_k) * gv, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hk = g.Hk, Hv = g.Hv, K = g.K, Km1 = g.K - 1, C = g.C_ch;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    const VtSmem lay = vt_smem(nm, gv, A.apart);
    const int early = vt_early(nm, A.apart);
    unsigned char *Bt = sm + lay.B, *Lt = sm + lay.L;
    bf* ws = reinterpret_cast<bf*>(sm + lay.w);
    int4* taps = reinterpret_cast<int4*>(sm + lay.taps);
    float* gate = reinterpret_cast<float*>(sm + lay.gate);
    float* glo = reinterpret_cast<float*>(sm + lay.lo);
    float* betas = reinterpret_cast<float*>(sm + lay.beta);
    float* eg = reinterpret_cast<float*>(sm + lay.eg);
    unsigned long long* line = reinterpret_cast<unsigned long long*>(sm + lay.line);
    unsigned long long* s_bad = reinterpret_cast<unsigned long long*>(sm + lay.bad);
    int* up = reinterpret_cast<int*>(sm + lay.up);
    // full, freed: state atoms; done: p and r; w_ready: w and e^G r in TMEM; t_ready: T; u_done, u_ready: u, rounded u;
    // o_done: o; o_read: o has left TMEM
    uint64_t *full = reinterpret_cast<uint64_t*>(sm + lay.bar), *freed = full + 2, *done = full + 4, *w_ready = full + 6,
             *t_ready = full + 8, *u_done = full + 10, *u_ready = full + 12, *o_done = full + 14, *o_read = full + 16, *bar_g = full + 18;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(full + 19);
    griddep_wait();  // launched with programmatic serialization
    griddep_launch_dependents();
    const int slot = J.slot_idx[b];
    const int64_t first = J.cu_nodes[b];
    const int64_t count = (int64_t)J.cu_nodes[b + 1] - first;
    if (slot < 0 || slot >= J.n_slots || first < 0 || count < 1 || count > J.max_nodes || first + count > J.n_nodes)
        return;
    const int n = (int)count;
    const int tcols = nm <= 16 ? 128 : (nm <= 32 ? 256 : 512);  // p and r of two v-heads, the Gram matrix, u of two v-heads
    const int halves = n > 32 ? 2 : 1;                          // warps that make T of a v-head
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(full + i, 1);
            mbar_init(freed + i, 1);
            mbar_init(done + i, 1);
            mbar_init(w_ready + i, kVtRows);
            mbar_init(t_ready + i, halves);
            mbar_init(u_done + i, 1);
            mbar_init(u_ready + i, kVtRows);
            mbar_init(o_done + i, 1);
            mbar_init(o_read + i, kVtRows);
        }
        mbar_init(bar_g, 1);
        fence_mbar_init();
        for (int i = 0; i < 5; ++i) s_bad[i] = 0ull;
    }
    if (warp == kVtWorkers) tc::alloc(tslot, tcols);
    const bf* xb = static_cast<const bf*>(J.x) + first * C;
    const bf* cb = static_cast<const bf*>(J.conv_pool) + (size_t)slot * Km1 * C;
    auto channel = [&](int what, int i) {  // first channel of k (0), q (1), v of v-head j0 + i (2)
        return (what == 0 ? Hk + h : (what == 1 ? h : 2 * Hk + j0 + i)) * D;
    };
    // the raw inputs of k and q, conv state first, into the places of A, P and v; those of v and z to L2
    bf* raw = reinterpret_cast<bf*>(sm + lay.A);
    for (int i = tid; i < (Km1 + n) * 32; i += kVtThreads) {
        const int row = i / 32, what = i / 16 % 2, c = i % 16 * 8;
        cp_async16(raw + row * 2 * D + what * D + c,
                   (row < Km1 ? cb + (size_t)row * C : xb + (size_t)(row - Km1) * C) + channel(what, 0) + c);
    }
    cp_async_commit();
    for (int node = warp; node < n; node += kVtThreads / 32) {
        const int jj = lane / 4, piece = lane % 4;
        if (jj < gv) tree_prefetch(piece < 2 ? xb + (size_t)node * C + channel(2, jj) + piece * 64
                                : static_cast<const bf*>(J.z) + ((size_t)(first + node) * Hv + j0 + jj) * D + (piece - 2) * 64);
    }
    // gates and parents; conv weights with the taps outside (a missing tap: 0).  What is read here is asked for before
    // any of it is used
    const int parent = tid < n ? J.parents[first + tid] : -1;
    const int jj0 = tid / nm, node0 = tid - jj0 * nm;  // the thread's first (v-head, node)
    const bool pair0 = jj0 < gv && node0 < n;
    const size_t at0 = (size_t)(first + (pair0 ? node0 : 0)) * Hv + j0 + (pair0 ? jj0 : 0);
    const int hv0 = j0 + (pair0 ? jj0 : 0);
    const bf a0 = static_cast<const bf*>(J.a)[at0], b0 = static_cast<const bf*>(J.b)[at0];
    const float alog0 = A.p.A_log[hv0], dt0 = A.p.dt_bias ? A.p.dt_bias[hv0] : 0.f;
    // weights of k, q and v-heads i0, i0 + 1 (what: from .. 3), by `nt` threads
    auto stage_weights = [&](int i0, int from, int nt) {
        constexpr int AHEAD = 2;
        const int end = (2 + min(2, gv - i0)) * D;
#pragma unroll 1
        for (int k0 = from * D + tid; k0 < end; k0 += AHEAD * nt) {
            bf w4[AHEAD][4];
#pragma unroll
            for (int e = 0; e < AHEAD; ++e) {
                const int k = min(k0 + e * nt, end - 1), what = k / D;
                const bf* src = static_cast<const bf*>(A.p.conv_w) + (size_t)(channel(min(what, 2), i0 + what - 2) + k % D) * K;
                if (K == 4) {
                    *reinterpret_cast<uint2*>(w4[e]) = __ldg(reinterpret_cast<const uint2*>(src));
                } else {
#pragma unroll
                    for (int m = 0; m < 4; ++m) w4[e][m] = m >= 4 - K ? src[m - (4 - K)] : __float2bfloat16_rn(0.f);
                }
            }
#pragma unroll
            for (int e = 0; e < AHEAD; ++e) {
                const int k = k0 + e * nt;
                if (k < end)
#pragma unroll
                    for (int m = 0; m < 4; ++m) ws[(k / D * 4 + m) * D + k % D] = w4[e][m];
            }
        }
    };
    stage_weights(0, 0, kVtThreads);
    if (tid < nm) {
        up[tid] = parent >= 0 && parent < tid ? parent : -1;
        line[tid] = 0ull;
    }
    for (int i = tid; i < nm * gv; i += kVtThreads) {  // (one turn, but for many v-heads)
        const int jj = i / nm, node = i - jj * nm;
        float la = 0.f, be = 0.f;
        if (i == tid) {
            if (pair0) gates(__bfloat162float(a0), __bfloat162float(b0), alog0, dt0, false, la, be);
        } else if (node < n) {
            const size_t at = (size_t)(first + node) * Hv + j0 + jj;
            gates(__bfloat162float(static_cast<const bf*>(J.a)[at]), __bfloat162float(static_cast<const bf*>(J.b)[at]),
                  A.p.A_log[j0 + jj], A.p.dt_bias ? A.p.dt_bias[j0 + jj] : 0.f, false, la, be);
        }
        gate[i] = tree_gate(la) * 1.4426950408889634f;
        betas[i] = be;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = *tslot, tgram = tm + 4 * nm, tu = tm + 5 * nm;
    const int atoms = 4 * gv;
    auto load = [&](int a) {  // atom a of the CTA's v-heads (4 each)
        mbar_arrive_expect_tx(full + (a & 1), kVtAtom);
        tma_tile_2d(sm + lay.S + (a & 1) * kVtAtom, &ts, (a & 3) * 32, (slot * Hv + j0 + (a >> 2)) * D, full + (a & 1));
    };
    if (tid == 32 * kVtWorkers)
        for (int i = 0; i < early; ++i) load(i);
    __syncwarp();
    if (early < 2) {  // the first v-head's state to L2
        const float* S = J.state_pool + ((size_t)slot * Hv + j0) * D * D;
        for (int i = tid; i < D * D / 32; i += kVtThreads) tree_prefetch(S + i * 32);
    }
    // the line of every node and the sums of log2 alpha along it; the conv taps' rows: the last tap is the node, then its
    // ancestors, then the conv state's rows, newest first
    for (int i = tid; i < n; i += kVtThreads) {
        unsigned long long m = 0;
        for (int at = i; at >= 0; at = up[at]) m |= 1ull << at;
        line[i] = m;
    }
    float sum[2] = {0.f, 0.f}, sum_lo[2] = {0.f, 0.f};  // (two (node, v-head) pairs to a thread at most: the launch sees to it)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = tid + e * kVtThreads, base = i / nm * nm;
        if (i < nm * gv)
            for (int at = i - base; at >= 0; at = up[at]) tree_add(sum[e], sum_lo[e], gate[base + at]);
    }
    if (tid >= kVtThreads - 64 && tid - (kVtThreads - 64) < n) {
        const int i = tid - (kVtThreads - 64);
        int at = i, row = Km1 - 1, t[4];
#pragma unroll
        for (int m = 3; m >= 0; --m) {
            const bool live = 3 - m < K;
            t[m] = !live ? Km1 + i : (at >= 0 ? Km1 + at : row--);
            if (live && at >= 0) at = up[at];
        }
        taps[i] = make_int4(t[0], t[1], t[2], t[3]);
    }
    cp_async_wait_all();
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // (read after the next barrier)
        const int i = tid + e * kVtThreads;
        if (i < nm * gv) {
            gate[i] = sum[e];
            glo[i] = sum_lo[e];
            eg[i] = tree_ex2(sum[e] + sum_lo[e]);
        }
    }
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {  // warp-wide; after a failure nothing waits any more
        if (ok) ok = vt_wait(bar, phase);
        return ok;
    };
    float* v = reinterpret_cast<float*>(sm + lay.v);
    const bf* bias = static_cast<const bf*>(A.p.conv_b);
    auto conv_v = [&](int i) {  // of v-head j0 + i, by the workers
        const int ch = channel(2, i) + 4 * lane;
#pragma unroll 1
        for (int i0 = NODES * warp; i0 < n; i0 += NODES * kVtWorkers)
            vt_conv_v<NODES>(reinterpret_cast<const unsigned char*>(xb + ch) - (size_t)Km1 * C * 2,
                             reinterpret_cast<const unsigned char*>(cb + ch), (uint32_t)C * 2u, taps,
                             reinterpret_cast<const uint2*>(ws + (2 + (i & 1)) * 4 * D), bias ? bias + ch : nullptr, K, i0, n, v);
    };
#pragma unroll 1
    for (int i0 = 2 * warp; i0 < n; i0 += 2 * (kVtWorkers + 1))
        vt_conv_kq<2>(smem_u32(raw + 4 * lane), taps, reinterpret_cast<const uint2*>(ws),
                      bias ? bias + channel(0, 0) + 4 * lane : nullptr, bias ? bias + channel(1, 0) + 4 * lane : nullptr, K, i0, n, Bt,
                      Lt, nm, g.q_scale, g.l2_eps);
    fence_proxy_async_smem();
    __syncthreads();  // [K^; Q^] is there
    if (warp == kVtWorkers) {
        // ---- products, and the state of each v-head in 4 atoms through a ring of two ---------
        const uint64_t db = tc::sdesc(tc::smem_addr(Bt)), ds = tc::sdesc(tc::smem_addr(sm + lay.S)),
                       dt = tc::sdesc(tc::smem_addr(sm + lay.A)), dp = tc::sdesc(tc::smem_addr(sm + lay.P));
        const uint32_t bstep = (uint32_t)(2 * nm * 128) >> 4, mstep = (uint32_t)(nm * 128) >> 4;
        const uint32_t id_n = tc::idesc_tf32(128, nm), id_2n = tc::idesc_tf32(128, 2 * nm);
        if (vt_elect()) {  // lanes are the rows of [K^; Q^] (what lies past them is never read), columns the keys
#pragma unroll 4
            for (int k = 0; k < 16; ++k)
                vt_mma(tgram, db + (k >> 2) * bstep + (k & 3) * 2, db + (k >> 2) * bstep + (k & 3) * 2, id_n, k > 0);
            // and what their rounding left out, times the values (bf16 is enough: 2^-9 of 2^-11), of either factor
            constexpr uint32_t id_bf = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(128 >> 4) << 24);
            const uint64_t dl = tc::sdesc(tc::smem_addr(Lt)), dx = dl + 2 * bstep;
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
                const uint32_t at = (k >> 2) * bstep + (k & 3) * 2;
                tc::mma_f16(tgram, dl + at, dx + at, id_bf | ((uint32_t)(nm >> 3) << 17), 1u);
                tc::mma_f16(tgram, dx + at, dl + at, id_bf | ((uint32_t)(nm >> 3) << 17), 1u);
            }
            tc::commit(bar_g);
        }
        __syncwarp();
        // whatever can go on does: a reload of the ring, an atom's product, u = w T^T or r += u P^T of a v-head
        auto ready = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, mbar_test(bar, (uint32_t)(phase & 1))); };
        int loaded = early, a = 0, fi = 0;
        bool u_issued = false;
        long long since = clock64();
#pragma unroll 1
        while (a < atoms || fi < gv) {
            bool moved = false;
            if (loaded < atoms && loaded < a + 2 && (loaded < 2 ? ready(bar_g, 0) : ready(freed + (loaded & 1), (loaded - 2) >> 1))) {
                if (lane == 0) load(loaded);
                __syncwarp();
                ++loaded;
                moved = true;
            }
            if (a < loaded && ready(full + (a & 1), a >> 1) &&
                ((a & 3) != 0 || a < 8 || ready(o_read + ((a >> 2) & 1), (a >> 3) - 1))) {  // o of v-head i - 2 has left TMEM
                const int i = a >> 2;
                tc::fence_after();
                if (vt_elect()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        vt_mma(tm + (i & 1) * 2 * nm, ds + (uint32_t)(((a & 1) * kVtAtom) >> 4) + k * 2,
                               db + (a & 3) * bstep + k * 2, id_2n, (a & 3) > 0 || k > 0);
                    tc::commit(freed + (a & 1));
                    if ((a & 3) == 3) tc::commit(done + (i & 1));
                }
                __syncwarp();
                ++a;
                moved = true;
            }
            if (fi < gv) {
                const int e = fi & 1, ph = fi >> 1;
                const uint32_t d = tm + e * 2 * nm, u = tu + e * nm;
                const uint64_t at = (uint64_t)(e * ((nm + 31) / 32)) * mstep;
                if (!u_issued ? ready(w_ready + e, ph) && ready(t_ready + e, ph) : ready(u_ready + e, ph)) {
                    tc::fence_after();
                    if (vt_elect()) {
#pragma unroll 1
                        for (int k = 0; k < (n + 7) / 8; ++k)
                            vt_mma_ta(u_issued ? d + nm : u, (u_issued ? u : d) + 8 * k,
                                      (u_issued ? dp : dt) + at + (k >> 2) * mstep + (k & 3) * 2, id_n, u_issued || k > 0);
                        tc::commit((u_issued ? o_done : u_done) + e);
                    }
                    __syncwarp();
                    if (u_issued) ++fi;
                    u_issued = !u_issued;
                    moved = true;
                }
            }
            const long long now = clock64();
            if (moved) {
                since = now;
            } else {
                if (__any_sync(0xffffffffu, now - since > kWaitLimitCycles)) {
                    ok = false;
                    break;
                }
                __nanosleep(40);
            }
        }
        if (!ok) {  // let the copies in flight land (bounded again); the others' waits give up by themselves
            for (int i = max(0, loaded - 2); i < loaded; ++i) mbar_wait(full + (i & 1), (uint32_t)((i >> 1) & 1));
            if (lane == 0) report_device_status(kDevWaitTimeout);
        }
    } else {
        const int tri = ((nm + 31) / 32) * nm * 128;  // bytes of A and of P of a v-head
#pragma unroll 1
        for (int i0 = 0; i0 < gv; i0 += 2) {  // v-heads i0 and i0 + 1
            const int two = min(2, gv - i0);
            if (i0 > 0) {  // (the v-heads before are finished: see the barrier at their end)
                stage_weights(i0, 2, 32 * kVtWorkers);
                if (tid < 5) s_bad[tid] = 0ull;
                named_bar_sync(1, 32 * kVtWorkers);
            }
            if (nm > 32) wait(bar_g, 0);  // (L reaches into v's place)
            conv_v(i0);
            // A and P from the Gram matrix: thread = row (a node's key, or its query), 8 columns at a time by the warps
            // of the row's quarter
            const int q4 = warp & 3, row = 32 * q4 + lane;
            if (32 * q4 < 2 * nm && wait(bar_g, 0)) {
                tc::fence_after();
                const bool is_q = row >= nm;
                const int i = is_q ? row - nm : row;
                const bool in = row < 2 * nm;
                const unsigned long long mine = in ? line[i] & ~(is_q ? 0ull : 1ull << i) : 0ull;
                const int ig = i0 * nm + (in ? i : 0);
                const float gi[2] = {gate[ig], gate[ig + (two - 1) * nm]}, li[2] = {glo[ig], glo[ig + (two - 1) * nm]};
                const float fi[2] = {is_q ? 1.f : betas[ig], is_q ? 1.f : betas[ig + (two - 1) * nm]};
                unsigned char* to = sm + (is_q ? lay.P : lay.A);
                float odd = 0.f;  // NaN from the first infinity or NaN on
#pragma unroll 1
                for (int c0 = 8 * (warp >> 2); c0 < nm; c0 += 8 * ((kVtWorkers - q4 + 3) / 4)) {
                    uint32_t r[8];
                    vt_ld8(tc::taddr(tgram, 32 * q4, c0), r);
                    tc::ld_wait();
                    const uint32_t m8 = (uint32_t)(mine >> c0) & 0xffu;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (e == two) break;
                        float x[8], gc[8], lc[8];
                        *reinterpret_cast<float4*>(gc) = *reinterpret_cast<const float4*>(gate + (i0 + e) * nm + c0);
                        *reinterpret_cast<float4*>(gc + 4) = *reinterpret_cast<const float4*>(gate + (i0 + e) * nm + c0 + 4);
                        *reinterpret_cast<float4*>(lc) = *reinterpret_cast<const float4*>(glo + (i0 + e) * nm + c0);
                        *reinterpret_cast<float4*>(lc + 4) = *reinterpret_cast<const float4*>(glo + (i0 + e) * nm + c0 + 4);
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            x[c] = (m8 >> c) & 1u ? tree_ex2((gi[e] - gc[c]) + (li[e] - lc[c])) * __uint_as_float(r[c]) * fi[e] : 0.f;
                            odd = fmaf(x[c], 0.f, odd);
                            if (is_q) x[c] = tc::to_tf32_rn(x[c]);
                        }
                        if (in) {
                            *reinterpret_cast<float4*>(vt_at(to + e * tri, nm, i, c0)) = make_float4(x[0], x[1], x[2], x[3]);
                            *reinterpret_cast<float4*>(vt_at(to + e * tri, nm, i, c0 + 4)) = make_float4(x[4], x[5], x[6], x[7]);
                        }
                    }
                    __syncwarp();
                }
                if (odd != 0.f) s_bad[4] = 1ull;
            }
            fence_proxy_async_smem();
            tc::fence_before();
            named_bar_sync(1, 32 * kVtWorkers);
            const int tw = kVtWorkers - 1 - warp;
            if (tw < two * halves) {
                // ---- T of v-head i0 + e in A's place, columns 32 half .. ------------------------------
                const int e = tw / halves, half = tw % halves, nb = (n + 15) / 16;
                unsigned char* T = sm + lay.A + e * tri;
                if (s_bad[4]) {  // 0 times an infinity or NaN is not 0: row by row, along the lines
                    if (half == 0) vt_lines(T, nm, n, line);
                    if (halves == 2) vt_pair_sync(e);
                } else {
                    vt_diag(T, nm, 2 * half, nb);
                    if (2 * half + 1 < nb) vt_below(T, nm, 32 * half + 16, 32 * half, 16, 16, 32 * half, -1);
                    if (halves == 2) {
                        vt_pair_sync(e);
                        vt_below(T, nm, 32, 0, 32, 16 * (nb - 2), 16 * half, e);
                        vt_pair_sync(e);
                    }
                }
                if (32 * half + lane < nm) {
                    uint32_t at = smem_u32(vt_at(T, nm, 32 * half, 32 * half + lane));
#pragma unroll 1
                    for (int r = 32 * half; r < 16 * nb; r += 8, at += 8 * 128) {  // the operand's rounding; above the diagonal are zeros
                        float t[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) t[k] = vt_ld1((at ^ (uint32_t)(k << 4)) + k * 128);
#pragma unroll
                        for (int k = 0; k < 8; ++k) vt_st1((at ^ (uint32_t)(k << 4)) + k * 128, tc::to_tf32_rn(t[k]));
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(t_ready + e);
            }
#pragma unroll 1
            for (int i = i0; i < i0 + two; ++i) {
                const int e = i & 1, ph = i >> 1;
                if (i > i0) {
                    conv_v(i);
                    named_bar_sync(1, 32 * kVtWorkers);
                }
                uint2 zr[kVtNorm];  // of the nodes below, kVtNorm at a time
                auto load_z = [&](int from) {
#pragma unroll
                    for (int q = 0; q < kVtNorm; ++q)
                        zr[q] = __ldg(reinterpret_cast<const uint2*>(
                                          static_cast<const bf*>(J.z) +
                                          ((size_t)(first + min(from + kVtWorkers * q, n - 1)) * Hv + j0 + i) * D) +
                                      lane);
                };
                if (warp >= kVtRows) load_z(warp);
                if (warp < kVtRows) {
                    // ---- thread = state row: w and e^G r, u rounded, then o in v's place --------------------
                    float* u = v + 32 * q4 + lane;
                    const int part = 8 * (warp >> 2);
                    const uint32_t tr = tc::taddr(tm, 32 * q4, e * 2 * nm), ur = tc::taddr(tu, 32 * q4, e * nm);
                    wait(done + e, ph);
                    tc::fence_after();
#pragma unroll 1
                    for (int c0 = part; c0 < n; c0 += 2 * kVtRows) {
                        uint32_t rk[8], rq[8];
                        vt_ld8(tr + c0, rk);
                        vt_ld8(tr + nm + c0, rq);
                        tc::ld_wait();
                        float be[8], f[8], w[8], wv[8], ro[8], odd = 0.f;
#pragma unroll
                        for (int c = 0; c < 8; c += 4) {
                            *reinterpret_cast<float4*>(be + c) = *reinterpret_cast<const float4*>(betas + i * nm + c0 + c);
                            *reinterpret_cast<float4*>(f + c) = *reinterpret_cast<const float4*>(eg + i * nm + c0 + c);
                        }
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            w[c] = be[c] * (u[(c0 + c) * D] - f[c] * __uint_as_float(rk[c]));
                            ro[c] = f[c] * __uint_as_float(rq[c]);
                            odd = fmaf(w[c], 0.f, odd);
                            wv[c] = tc::to_tf32_rn(w[c]);
                        }
                        if (odd != 0.f || c0 + 8 > n) {
                            // T and P are 0 off the line, but 0 times an infinity or NaN is not: those are added below
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const bool fine = isfinite(w[c]);
                                if (!fine && c0 + c < n) {
                                    atomicOr(s_bad + e, 1ull << (c0 + c));
                                    u[(c0 + c) * D] = w[c];
                                }
                                if (!fine || c0 + c >= n) wv[c] = 0.f;
                            }
                        }
                        __syncwarp();
                        vt_st8(tr + c0, wv);
                        vt_st8(tr + nm + c0, ro);
                    }
                    tc::st_wait();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(w_ready + e);
                    load_z(warp);
                    named_bar_sync(4, 32 * kVtRows);
                    const unsigned char *Tm = sm + lay.A + e * tri, *Pm = sm + lay.P + e * tri;
                    // columns `cols` plus the bad nodes' part, which the product left out: (T or P) times (w or u)
                    auto add_bad = [&](uint32_t cols, const unsigned char* m, unsigned long long bad) {
#pragma unroll 1
                        for (int c0 = part; c0 < n; c0 += 2 * kVtRows) {
                            uint32_t r[8];
                            float x[8];
                            vt_ld8(cols + c0, r);
                            tc::ld_wait();
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                x[c] = __uint_as_float(r[c]);
                                const int node = min(c0 + c, n - 1);
                                for (unsigned long long left = bad & line[node]; left; left &= left - 1) {
                                    const int a = __ffsll((long long)left) - 1;
                                    // (finite here: it was in the product)
                                    if (!isfinite(u[a * D])) x[c] = fmaf(*vt_at(const_cast<unsigned char*>(m), nm, node, a), u[a * D], x[c]);
                                }
                            }
                            __syncwarp();
                            vt_st8(cols + c0, x);
                        }
                        tc::st_wait();
                        named_bar_sync(4, 32 * kVtRows);
                    };
                    wait(u_done + e, ph);
                    tc::fence_after();
                    if (s_bad[e]) add_bad(ur, Tm, s_bad[e]);  // (the same for all of these warps)
#pragma unroll 1
                    for (int c0 = 2 * part; c0 < n; c0 += 4 * kVtRows) {
                        uint32_t r[16];
                        float x[16], odd = 0.f;
                        vt_ld8(ur + c0, r);
                        vt_ld8(ur + c0 + 8, r + 8);
                        tc::ld_wait();
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            odd = fmaf(__uint_as_float(r[c]), 0.f, odd);
                            x[c] = tc::to_tf32_rn(__uint_as_float(r[c]));
                        }
                        if (odd != 0.f) {
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                if (isfinite(__uint_as_float(r[c]))) continue;
                                x[c] = 0.f;
                                if (c0 + c >= n) continue;
                                atomicOr(s_bad + 2 + e, 1ull << (c0 + c));
                                u[(c0 + c) * D] = __uint_as_float(r[c]);
                            }
                        }
                        __syncwarp();
                        vt_st8(ur + c0, x);
                        vt_st8(ur + c0 + 8, x + 8);
                    }
                    tc::st_wait();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(u_ready + e);
                    named_bar_sync(4, 32 * kVtRows);
                    wait(o_done + e, ph);
                    tc::fence_after();
                    if (s_bad[2 + e]) add_bad(tr + nm, Pm, s_bad[2 + e]);
#pragma unroll 1
                    for (int c0 = 2 * part; c0 < n; c0 += 4 * kVtRows) {
                        uint32_t ro[16];
                        vt_ld8(tr + nm + c0, ro);
                        vt_ld8(tr + nm + c0 + 8, ro + 8);
                        tc::ld_wait();
#pragma unroll
                        for (int c = 0; c < 16; ++c) u[(c0 + c) * D] = __uint_as_float(ro[c]);  // (nm rows of room)
                    }
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_read + e);  // this v-head's columns are free
                }
                named_bar_sync(1, 32 * kVtWorkers);
                // gated RMSNorm, a warp per node, kVtNorm at once, four channels to a lane
                const uint2 nw = __ldg(reinterpret_cast<const uint2*>(A.p.norm_w) + lane);
                const float2 w01 = vt_two(nw.x), w23 = vt_two(nw.y);
#pragma unroll 1
                for (int n0 = warp; n0 < n; n0 += kVtNorm * kVtWorkers) {
                    if (n0 > warp) load_z(n0);
                    float4 o[kVtNorm];
                    float ss[kVtNorm];
#pragma unroll
                    for (int q = 0; q < kVtNorm; ++q) {
                        o[q] = *reinterpret_cast<const float4*>(v + min(n0 + kVtWorkers * q, n - 1) * D + 4 * lane);
                        ss[q] = fmaf(o[q].x, o[q].x, fmaf(o[q].y, o[q].y, fmaf(o[q].z, o[q].z, o[q].w * o[q].w)));
                    }
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                        for (int q = 0; q < kVtNorm; ++q) ss[q] += __shfl_xor_sync(0xffffffffu, ss[q], off);
#pragma unroll
                    for (int q = 0; q < kVtNorm; ++q) {
                        const int node = n0 + kVtWorkers * q;
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
                if (i + 1 < gv) named_bar_sync(1, 32 * kVtWorkers);  // o is read: its place takes the next v
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kVtWorkers) tc::dealloc(tm, tcols);
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

template <int CTAS>
cudaError_t launch_verify_ctas(const CUtensorMap& map, const VtArgs& A, cudaStream_t st) {
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t e = raise_smem_limit(k_tree_verify_tc<CTAS>, 227 * 1024, smem_set);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_tree_verify_tc<CTAS>, dim3((unsigned)(A.g.Hv / A.gv), (unsigned)A.job.B), dim3(kVtThreads),
                      (size_t)vt_smem(A.nm, A.gv, A.apart).total + 1024, st, map, A);
}

cudaError_t launch_verify_tc(const Geom& g, const LayerParams& p, const TreeJob& job, cudaStream_t st) {
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
    VtArgs A{g, p, job, (job.max_nodes + 15) / 16 * 16, g.G, 0};
    // Few trees: a CTA per v-head (us, 16 / 32 heads: one tree of 8 nodes 9.4 against 12.3, 8 of 16 nodes 12.5 against
    // 14.1).  From a CTA per SM on: all v-heads of a k-head, which share its conv and Gram matrix (16 of 16 nodes 18.8
    // against 22.4, 64 of 32 nodes 81 against 105), or as many as shared memory and two (node, v-head) pairs a thread allow
    if ((long)job.B * g.Hk < sm_count()) A.gv = 1;
    while (vt_smem(A.nm, A.gv, 0).total + 1024 > 227 * 1024 || A.nm * A.gv > 2 * kVtThreads || A.gv > 8 || A.g.G % A.gv) --A.gv;
    // L in a place of its own while all CTAs are resident all the same: the state is on its way from the start then (us: 8 of 16
    // nodes 12.5 against 13.2, 16 of 16 nodes 18.8 against 19.2)
    const long per_sm = ((long)job.B * (g.Hv / A.gv) + sm_count() - 1) / sm_count();
    A.apart = A.nm <= 32 && per_sm <= 2 && per_sm * (vt_smem(A.nm, A.gv, 1).total + 2048) <= 228 * 1024;
    // Trees of up to 16 nodes leave shared memory for a third CTA on an SM: with fewer registers each, faster once more than
    // two have work (us, 16 / 32 heads: 64 trees of 8 nodes 49 against 56; one tree 9.6 against 9.4; trees of up to 32 nodes,
    // where shared memory holds two, 86 against 81)
    if (A.nm <= 16 && (long)job.B * (g.Hv / A.gv) > 2L * sm_count()) return launch_verify_ctas<3>(map, A, st);
    return launch_verify_ctas<2>(map, A, st);
}

// ---- commit ---------------------------------------------------------------------
// One CTA per (v-head, sequence), a cluster per k-head.  A warp holds D / 8 state rows in registers
// through all rows of the path (a state row's update touches no other row), 8 lanes to a row as in
// k_tree_verify, so the state is read once and written once, and shared memory holds only
// the inputs, k and v of a chunk of path rows at a time.  Bound by DRAM latency at two CTAs an SM (HBM half busy).  The state
// is asked for last: the short dependent loads of the inputs stand in line behind it otherwise, and the SM's other CTA keeps HBM
// busy meanwhile
// (64 sequences of up to 6 rows, 48 v-heads of 128 x 128: 86 us, 4.8 TB/s; 89 with the state asked for before k and v are
// made, 96 before the inputs, 98 by a bulk copy at the start, 92 with a prefetch to L2 a wave ahead).
// The G CTAs of a k-head read the same conv rows of k, which one of them replaces: the cluster barrier stands between.
template <typename TA>
constexpr int kComChunk = sizeof(TA) == 2 ? 16 : 8;

struct CommitArgs {
    Geom g;
    LayerParams p;
    TreeCommitJob job;
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
    if (slot < 0 || slot >= J.n_slots || first < 0 || count < 1 || count > J.max_rows || first + count > J.n_rows)
        return;  // the whole cluster shares b
    const int l8 = lane & 7, grp = lane >> 3, row0 = warp * (D / 8) + grp;  // state row r * 4 + group, columns 4 l8 + 32 c
    float* Sg = J.state_pool + (((size_t)slot * Hv + j) * D + row0) * D + 4 * l8;
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
    // the raw inputs of the rows t0 .., all on their way at once (through shared memory: the state has the registers):
    // input p of the sequence is row p of the conv state, then the path's rows
    auto stage = [&](int t0) {
        constexpr int PER = D * (int)sizeof(TA) / 16;  // 16-byte pieces of a row's head
        const int m = min(kComRows, n - t0);
        for (int i = tid; i < (m + Km1) * 3 * PER; i += kTreeThreads) {
            const int row = i / (3 * PER), kind = i / PER % 3, c = i % PER * (16 / (int)sizeof(TA)), p = t0 + row;
            cp_async16(&hs[row][kind][c], (p < Km1 ? cp + (size_t)p * C : x + (size_t)rows[p - Km1] * C) + channel(kind) + c);
        }
        cp_async_commit();
    };
    stage(0);
    {
        const bool direct = g.flags & kFlagGatesDirect;
        for (int t = tid - (kTreeThreads - 64); t >= 0 && t < n; t += 64) {
            float gl, beta;
            gates(L::ld(J.a, (size_t)rows[t] * Hv + j), L::ld(J.b, (size_t)rows[t] * Hv + j), direct ? 0.f : A.p.A_log[j],
                  !direct && A.p.dt_bias ? A.p.dt_bias[j] : 0.f, direct, gl, beta);
            alpha_s[t] = expf(gl);
            beta_s[t] = beta;
        }
    }
    float4 S[RL][RL];
    for (int t0 = 0; t0 < n; t0 += kComRows) {
        const int m = min(kComRows, n - t0);
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
        if (t0 == 0) {
#pragma unroll
            for (int r = 0; r < RL; ++r)
#pragma unroll
                for (int c = 0; c < RL; ++c) S[r][c] = *reinterpret_cast<const float4*>(Sg + (size_t)r * 4 * D + 32 * c);
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
        if (t0 + kComRows < n) {
            __syncthreads();  // ks, vs and the inputs are read
            stage(t0 + kComRows);
        }
    }
#pragma unroll
    for (int r = 0; r < RL; ++r)
#pragma unroll
        for (int c = 0; c < RL; ++c) *reinterpret_cast<float4*>(Sg + (size_t)r * 4 * D + 32 * c) = S[r][c];
    // the new conv state: the last K - 1 raw inputs, bit for bit, from shared memory
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
    // d = 128, bf16: on the tensor cores (us against the CUDA cores: 64 trees of up to 32 nodes 81, 155; one of 16 nodes
    // 10.4, 14.5; of 12 10.5, 13.0; 16 of 8 16.0, 21.2), but for trees of up to 8 nodes while every (tree, v-head) has an SM: the
    // phases are longer than the work then (one tree of 8 nodes 9.1 on the CUDA cores, 9.4; of 4 6.5, 9.3; of 1 5.1, 8.9;
    // 4 trees of 8 9.1, 9.9)
    const bool few = job.max_nodes <= 8 && (long)job.B * g.Hv <= sm_count();
    if (g.D == 128 && g.act_bf16 && g.flags == 0 && !few) return launch_verify_tc(g, p, job, st);
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
