// Eviction from the paged caches by accumulated attention weight: which
// positions of each sequence stay, and the move of their rows to the front.
#pragma once
#include "common.cuh"

namespace dsa {
namespace cache_evict {

// Order key of a weight: larger is kept first; a NaN ranks with -inf.
__device__ __forceinline__ uint32_t mass_key(float v) { return score_key(v == v ? v : -INFINITY); }

constexpr int kSelectThreads = 1024;
constexpr int kMaxLen = 1 << 30;       // positions of a sequence
constexpr int kMaxRowBytes = 4096;     // bytes of a cache row that compaction moves

// Block-wide exclusive sum of one int per thread; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

// One CTA per sequence: the positions that stay, ascending. The free places
// (keep - sinks - recent) go to the largest weights of the unprotected
// positions [sinks, n - recent), ties to the lower position: a radix select on
// the order key's four bytes finds the last key that stays and how many of
// its equals do.
__global__ void __launch_bounds__(kSelectThreads)
cache_evict_select_kernel(const float* __restrict__ mass, long long ld, const int* __restrict__ seq_len,
                          int max_len, int keep, int sinks, int recent, int* __restrict__ keep_idx,
                          int* __restrict__ new_len)
{
    __shared__ int hist[256], wsum[32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int n = max(0, min(seq_len[b], max_len));
    const float* row = mass + b * ld;
    int* idx = keep_idx + (size_t)b * keep;
    if (tid == 0) new_len[b] = min(n, keep);
    if (n <= keep) {
        for (int j = tid; j < keep; j += kSelectThreads) idx[j] = j < n ? j : -1;
        return;
    }
    const int lo = sinks, hi = n - recent;   // unprotected
    if (tid == 0) {
        s_prefix = 0;
        s_need = keep - sinks - recent;
    }
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t prefix = s_prefix;
        for (int s = lo + tid; s < hi; s += kSelectThreads) {
            const uint32_t k = mass_key(row[s]);
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int need = s_need, d = 255;
            for (; d > 0 && hist[d] < need; --d) need -= hist[d];
            s_prefix = prefix | ((uint32_t)d << shift);
            s_need = need;
        }
        __syncthreads();
    }
    // keys above `cut` stay, and the first `ties` of its equals
    const uint32_t cut = s_prefix;
    int ties = s_need, at = 0;
    for (int s0 = 0; s0 < n; s0 += kSelectThreads) {
        const int s = s0 + tid;
        bool stays = s < n && (s < lo || s >= hi), eq = false;
        if (s >= lo && s < hi) {
            const uint32_t k = mass_key(row[s]);
            stays = k > cut;
            eq = k == cut;
        }
        int n_eq, n_stay;
        const int before = block_scan(eq ? 1 : 0, wsum, &n_eq);
        if (eq && before < ties) stays = true;
        ties -= min(ties, n_eq);
        const int place = block_scan(stays ? 1 : 0, wsum, &n_stay);
        if (stays) idx[at + place] = s;
        at += n_stay;
    }
}

constexpr int kCompactThreads = 256;

// Rows of `bytes` bytes (a multiple of 16) moved in place: row idx[j] of the
// sequence to row j, j < new_len. As idx ascends and idx[j] >= j, a block of
// rows can be written once it and the blocks before it are read. One CTA per
// (sequence, slice of the row).
__global__ void __launch_bounds__(kCompactThreads)
cache_compact_kernel(uint8_t* __restrict__ rows, int row_bytes, int slice, const PagedRows pg,
                     const int* __restrict__ keep_idx, int keep, const int* __restrict__ new_len)
{
    const int b = blockIdx.x, c0 = blockIdx.y * slice;
    const int pieces = min(slice, row_bytes - c0) / 16;
    const int per = kCompactThreads / pieces;   // rows a block of threads holds
    const int r = threadIdx.x / pieces, piece = threadIdx.x % pieces;
    const int S = pg.max_pages * pg.page_size;
    const int* bt = pg.block_table + (size_t)b * pg.max_pages;
    const int* idx = keep_idx + (size_t)b * keep;
    const int m = min(min(new_len[b], keep), S);
    auto place = [&](int s) -> uint4* {
        const int page = bt[s / pg.page_size];
        if ((unsigned)page >= (unsigned)pg.num_pages) return nullptr;
        return reinterpret_cast<uint4*>(rows + ((size_t)page * pg.page_size + s % pg.page_size) * row_bytes + c0) + piece;
    };
    for (int j0 = 0; j0 < m; j0 += per) {
        const int j = j0 + r;
        uint4 v;
        uint4* to = nullptr;
        if (r < per && j < m) {
            const int s = idx[j];
            if (s > j && s < S) {
                const uint4* from = place(s);
                to = place(j);
                if (from && to)
                    v = *from;
                else
                    to = nullptr;
            }
        }
        __syncthreads();
        if (to) *to = v;
        __syncthreads();
    }
}

// The weights moved likewise; the places behind the last kept one are zeroed.
__global__ void __launch_bounds__(kCompactThreads)
cache_compact_mass_kernel(float* __restrict__ mass, int S, const int* __restrict__ keep_idx, int keep,
                          const int* __restrict__ new_len)
{
    float* row = mass + (size_t)blockIdx.x * S;
    const int* idx = keep_idx + (size_t)blockIdx.x * keep;
    const int m = max(0, min(min(new_len[blockIdx.x], keep), S));
    for (int j0 = 0; j0 < m; j0 += kCompactThreads) {
        const int j = j0 + threadIdx.x;
        float v = 0.f;
        bool moves = false;
        if (j < m) {
            const int s = idx[j];
            moves = s > j && s < S;
            if (moves) v = row[s];
        }
        __syncthreads();
        if (moves) row[j] = v;
        __syncthreads();
    }
    for (int j = m + threadIdx.x; j < S; j += kCompactThreads) row[j] = 0.f;
}

}  // namespace cache_evict
}  // namespace dsa
