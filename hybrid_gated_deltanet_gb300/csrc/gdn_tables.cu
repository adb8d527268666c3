// gdn_tables.cu -- the bookkeeping of a paged cache on the device: pages and row
// maps from request lengths (gdn_page_tables), and K and V rows into their pages by
// such a map (gdn_attn_append).
#include <cuda_bf16.h>

#include <algorithm>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_tma.cuh"

namespace gdn {
namespace {

// ---- pages and row maps -------------------------------------------------------
// need[b] = ceil((ctx + new) / page) - ceil(ctx / page); sequence b is granted when the
// running sum of need (and of new) up to and including b fits, so the j-th new page of b is
// free_pages[head + sum of need before b + j]: two prefix sums decide everything.
// Every CTA repeats them (1024 sequences at a time, a few KB from L2) instead of
// handing them over through memory, and then writes its own share of the rows and
// pages: one launch, no workspace, no wait between CTAs.  Old table entries are read
// only below ceil(ctx / page) and new ones written only from there on, so the table
// is updated in place without a race.  Latency-bound: the work is a few bytes a row (64 paths 4.9 us, 20 prompts of up to
// 30000 tokens 6.1 us).
constexpr int kTabThreads = 512;
constexpr int kTabChunk = 1024;  // sequences per scan step: 2 per thread

struct Two {
    long long pages, rows;
};

// inclusive sums over the block's threads
__device__ __forceinline__ Two block_scan(Two v, Two* warp_tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long p = __shfl_up_sync(0xffffffffu, v.pages, off), r = __shfl_up_sync(0xffffffffu, v.rows, off);
        if (lane >= off) {
            v.pages += p;
            v.rows += r;
        }
    }
    if (lane == 31) warp_tot[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        v.pages += warp_tot[w].pages;
        v.rows += warp_tot[w].rows;
    }
    return v;
}

// last i in [0, n) with start[i] <= at (start is non-decreasing, start[0] <= at); of
// equal starts the last, which is the one that is not empty
__device__ __forceinline__ int owner_of(const int* start, int n, unsigned at) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((unsigned)start[mid] <= at) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads) k_page_tables(const __grid_constant__ TablesJob J) {
    __shared__ Two tot[kTabThreads / 32], carry_s;
    __shared__ int s_row[kTabChunk + 1], s_page[kTabChunk + 1];  // first row and first new page of each sequence
    __shared__ int s_ctx[kTabChunk];
    griddep_wait();  // launched with programmatic serialization
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int head = J.head[0];
    const long long room = head < 0 ? 0 : (long long)J.n_free - head;
    Two asked{0, 0};              // need and new of every sequence before the chunk
    int rows_done = 0, used = 0;  // granted rows and pages before the chunk
    for (int b0 = 0; b0 < J.B; b0 += kTabChunk) {
        const int nb = min(kTabChunk, J.B - b0);
        long long need[2], add[2];
        Two mine{0, 0};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * tid + e;
            need[e] = add[e] = 0;
            if (i < nb) {
                const long long c = J.ctx_lens[b0 + i], n = J.new_lens[b0 + i];
                s_ctx[i] = (int)c;
                const bool fits = c >= 0 && n >= 0 && c + n <= (long long)J.max_pages * J.page &&
                                  (J.path == nullptr || n <= J.path_len);
                if (fits) {
                    need[e] = (c + n + J.page - 1) / J.page - (c + J.page - 1) / J.page;
                    add[e] = n;
                }
            }
            mine.pages += need[e];
            mine.rows += add[e];
        }
        const Two incl = block_scan(mine, tot);
        Two before{asked.pages + incl.pages - mine.pages, asked.rows + incl.rows - mine.rows};
        Two granted{0, 0};
        long long g_need[2], g_add[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            before.pages += need[e];  // now inclusive of sequence 2 tid + e
            before.rows += add[e];
            const bool ok = add[e] > 0 && (need[e] == 0 || before.pages <= room) && before.rows <= J.n_rows;
            g_need[e] = ok ? need[e] : 0;
            g_add[e] = ok ? add[e] : 0;
            granted.pages += g_need[e];
            granted.rows += g_add[e];
        }
        if (tid == kTabThreads - 1) carry_s = Two{asked.pages + incl.pages, asked.rows + incl.rows};
        __syncthreads();  // tot may be used again
        const Two done = block_scan(granted, tot);
        int row = rows_done + (int)(done.rows - granted.rows), pg = used + (int)(done.pages - granted.pages);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * tid + e;
            s_row[i] = row;
            s_page[i] = pg;
            if (blockIdx.x == 0 && i < nb) J.cu_rows[b0 + i] = row;
            row += (int)g_add[e];
            pg += (int)g_need[e];
        }
        if (tid == kTabThreads - 1) {
            s_row[kTabChunk] = row;
            s_page[kTabChunk] = pg;
        }
        __syncthreads();
        asked = carry_s;
        const int row_end = s_row[kTabChunk], page_end = s_page[kTabChunk];
        // the chunk's new pages (counters without a sign: up to 2^31 - 1 of them, and a grid's stride more)
        for (unsigned k = used + blockIdx.x * kTabThreads + tid; k < (unsigned)page_end; k += gridDim.x * kTabThreads) {
            const int i = owner_of(s_page, nb, k);
            const long long col = ((long long)s_ctx[i] + J.page - 1) / J.page + (int)(k - s_page[i]);
            J.block_table[(size_t)(b0 + i) * J.max_pages + col] = J.free_pages[head + (int)k];
        }
        // the chunk's rows
        for (unsigned k = rows_done + blockIdx.x * kTabThreads + tid; k < (unsigned)row_end; k += gridDim.x * kTabThreads) {
            const int i = owner_of(s_row, nb, k), at = (int)(k - s_row[i]);
            const unsigned pos = (unsigned)s_ctx[i] + (unsigned)at, page = (unsigned)J.page;
            const unsigned pc = pos / page, old = ((unsigned)s_ctx[i] + page - 1) / page;
            const int id = pc >= old ? J.free_pages[head + s_page[i] + (int)(pc - old)]
                                     : J.block_table[(size_t)(b0 + i) * J.max_pages + pc];
            J.slot_map[k] = id >= 0 && id < J.n_pages ? (int64_t)id * page + pos % page : -1;
            if (J.src_rows) {
                const int first = J.cu_nodes[b0 + i], n = J.cu_nodes[b0 + i + 1] - first;
                const int node = J.path[(size_t)(b0 + i) * J.path_len + at];
                J.src_rows[k] = node >= 0 && node < n ? first + node : -1;
            }
        }
        rows_done = row_end;
        used = page_end;
        __syncthreads();  // the chunk's tables are read
    }
    for (unsigned k = rows_done + blockIdx.x * kTabThreads + tid; k < (unsigned)J.n_rows; k += gridDim.x * kTabThreads) {
        J.slot_map[k] = -1;
        if (J.src_rows) J.src_rows[k] = -1;
    }
    if (blockIdx.x == 0 && tid == 0) {
        J.cu_rows[J.B] = rows_done;
        J.head_out[0] = head + used;
    }
}

// ---- K and V rows into their pages --------------------------------------------
// thread = 16 bytes of K and the same 16 of V, kAppUnroll of them a grid apart, so that
// 2 kAppUnroll loads are in flight: a copy, bound by HBM (65536 rows of 2 heads of 256: 44 us, 6.1 TB/s) or by the
// launch when short (300 rows: 2.4 us)
constexpr int kAppThreads = 256;
constexpr int kAppUnroll = 2;

__global__ void __launch_bounds__(kAppThreads) k_append_rows(const __grid_constant__ AppendJob J) {
    griddep_wait();
    griddep_launch_dependents();
    const int per_head = J.D / 8, per_row = J.Hkv * per_head;  // 16-byte pieces
    const int64_t total = J.n_rows * per_row, step = (int64_t)gridDim.x * kAppThreads;
    const uint4* ks = static_cast<const uint4*>(J.k_new);
    const uint4* vs = static_cast<const uint4*>(J.v_new);
    uint4* kd = static_cast<uint4*>(J.k_pool);
    uint4* vd = static_cast<uint4*>(J.v_pool);
    const int64_t n_slots = (int64_t)J.n_pages * J.page;
    for (int64_t i0 = blockIdx.x * (int64_t)kAppThreads + threadIdx.x; i0 < total; i0 += kAppUnroll * step) {
        uint4 k[kAppUnroll], v[kAppUnroll];
        int64_t dst[kAppUnroll];
#pragma unroll
        for (int e = 0; e < kAppUnroll; ++e) {
            const int64_t i = i0 + e * step;
            dst[e] = -1;
            if (i >= total) continue;
            const int64_t row = i / per_row;
            const int c = (int)(i - row * per_row);
            const int64_t slot = J.slot_map[row];
            const int64_t src = J.src_rows ? J.src_rows[row] : row;
            if (slot < 0 || slot >= n_slots || src < 0 || src >= J.n_src) continue;
            const int64_t page = slot / J.page, at = slot - page * J.page;
            k[e] = ks[src * per_row + c];
            v[e] = vs[src * per_row + c];
            dst[e] = ((page * J.Hkv + c / per_head) * J.page + at) * per_head + c % per_head;
        }
#pragma unroll
        for (int e = 0; e < kAppUnroll; ++e) {
            if (dst[e] < 0) continue;
            kd[dst[e]] = k[e];
            vd[dst[e]] = v[e];
        }
    }
}

}  // namespace

cudaError_t launch_page_tables(const TablesJob& job, cudaStream_t st) {
    // about 2 rows a thread, at most one CTA per SM
    const int64_t want = ((int64_t)job.n_rows + 2 * kTabThreads - 1) / (2 * kTabThreads);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(want, sm_count()));
    return launch_pdl(k_page_tables, dim3(grid), dim3(kTabThreads), 0, st, job);
}

cudaError_t launch_append(const AppendJob& job, cudaStream_t st) {
    if (job.n_rows == 0 || job.n_src == 0) return cudaSuccess;
    const int64_t total = job.n_rows * (job.Hkv * (job.D / 8));
    const int64_t want = (total + kAppThreads * kAppUnroll - 1) / (kAppThreads * kAppUnroll);
    const int grid = (int)std::min<int64_t>(want, (int64_t)sm_count() * 32);
    return launch_pdl(k_append_rows, dim3(grid), dim3(kAppThreads), 0, st, job);
}

}  // namespace gdn
