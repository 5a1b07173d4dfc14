// Eviction from the paged caches by accumulated attention weight: which
// positions of each sequence stay, and the move of their rows to the front.
#pragma once
#include "common.cuh"
#include "sm100.cuh"

namespace dsa {
namespace cache_evict {

using sm100::cluster_ctarank;
using sm100::cluster_sync;
using sm100::mapa;
using sm100::smem_u32;

constexpr int kMaxLen = 1 << 30;       // positions of a sequence
constexpr int kMaxRowBytes = 4096;     // bytes of a cache row that compaction moves

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}

// ------------------------------------------------------------------ select

// Order key of a weight: larger is kept first; a NaN ranks with -inf.
__device__ __forceinline__ uint32_t mass_key(float v) { return score_key(v == v ? v : -INFINITY); }

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelRound = 16384;                     // positions a CTA holds in shared memory
constexpr int kBins = 2048;
constexpr int kSelMaxCluster = 8;
constexpr int kSelSmem = kSelRound * 4 + kBins * 4;

// Block-wide exclusive sum of one int per thread.
__device__ __forceinline__ int block_scan(int v, int* warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w)
        if (w < warp) before += warp_sums[w];
    return before + x - v;
}

// One cluster per sequence; its CTAs, and their warps, take contiguous shares
// of the positions. The free places (keep - sinks - recent) go to the largest
// weights of the unprotected positions [sinks, n - recent), ties to the lower
// position: a radix select over the order key's bits, 11 + 11 + 10, finds the
// last key that stays and how many of its equals do; each digit's histogram
// is summed over the cluster's shared memory. Up to 16384 positions per CTA
// the order keys stay in shared memory (three CTAs a SM; in registers only
// one of 1024 threads fits, and 64 sequences took four rounds of the card: 151
// us against 40); longer sequences read the weights again for each digit.
__global__ void __launch_bounds__(kSelThreads, 3)
cache_evict_select_kernel(const float* __restrict__ mass, long long ld, const int* __restrict__ seq_len,
                          int max_len, int keep, int sinks, int recent, int* __restrict__ keep_idx,
                          int* __restrict__ new_len)
{
    extern __shared__ __align__(16) uint32_t sel_smem[];
    uint32_t* held = sel_smem;                                      // [kSelRound] order keys
    int* hist = reinterpret_cast<int*>(sel_smem + kSelRound);       // [kBins]
    __shared__ int wsum[kSelWarps];
    __shared__ int s_digit, s_need;
    __shared__ int counts[2];          // this CTA's positions above the cut (or protected), and equal to it
    __shared__ int w_stay[kSelWarps], w_eq[kSelWarps];
    const int rank = (int)cluster_ctarank(), size = (int)cluster_size();
    const int b = (int)(blockIdx.x / size), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = max(0, min(seq_len[b], max_len));
    const float* row = mass + b * ld;
    int* idx = keep_idx + (size_t)b * keep;
    if (rank == 0 && tid == 0) new_len[b] = min(n, keep);
    if (n <= keep) {                   // the whole cluster: no barrier is left behind
        for (int j = rank * kSelThreads + tid; j < keep; j += size * kSelThreads) idx[j] = j < n ? j : -1;
        return;
    }
    const int lo = sinks, hi = n - recent;   // unprotected
    // this CTA's share [c0, c1) of the positions
    const int share = (int)(((long long)n + (long long)size * 4 - 1) / ((long long)size * 4)) * 4;
    const int c0 = min(n, rank * share), c1 = min(n, c0 + share);
    const bool in_smem = share <= kSelRound;
    for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
    if (in_smem) {
        if ((reinterpret_cast<uintptr_t>(row + c0) & 15u) == 0) {
#pragma unroll 8
            for (int s = c0 + 4 * tid; s < c1; s += 4 * kSelThreads) {
                float4 v;
                if (s + 4 <= c1) {
                    v = __ldg(reinterpret_cast<const float4*>(row + s));
                } else {
                    v.x = row[s];
                    v.y = s + 1 < c1 ? row[s + 1] : 0.f;
                    v.z = s + 2 < c1 ? row[s + 2] : 0.f;
                    v.w = 0.f;
                }
                *reinterpret_cast<uint4*>(held + (s - c0)) = make_uint4(mass_key(v.x), mass_key(v.y), mass_key(v.z),
                                                                       mass_key(v.w));
            }
        } else {
#pragma unroll 8
            for (int s = c0 + tid; s < c1; s += kSelThreads) held[s - c0] = mass_key(row[s]);
        }
    }
    __syncthreads();
    auto key_at = [&](int s) -> uint32_t { return in_smem ? held[s - c0] : mass_key(row[s]); };
    uint32_t prefix = 0, known = 0;          // digits found so far and their bits
    int need = keep - sinks - recent;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
        const int s1 = min(c1, hi);
#pragma unroll 8
        for (int s = max(c0, lo) + tid; s < s1; s += kSelThreads) {
            const uint32_t k = key_at(s);
            if ((k & known) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
        }
        cluster_sync();
        // bins from the top down, four per thread (bin index 4 tid' + 3 .. 4 tid'), summed over the cluster
        const int top = bins - 4 - 4 * tid;
        int v[4] = {0, 0, 0, 0};
        if (top >= 0) {
            uint4 part[kSelMaxCluster];
#pragma unroll
            for (int c = 0; c < kSelMaxCluster; ++c)
                if (c < size) part[c] = sm100::ld_cluster_v4(mapa(smem_u32(hist + top), (uint32_t)c));
#pragma unroll
            for (int c = 0; c < kSelMaxCluster; ++c)
                if (c < size) {
                    v[0] += (int)part[c].w;
                    v[1] += (int)part[c].z;
                    v[2] += (int)part[c].y;
                    v[3] += (int)part[c].x;
                }
        }
        int before = block_scan(v[0] + v[1] + v[2] + v[3], wsum);
        if (top >= 0 && before < need) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (before < need && before + v[e] >= need) {
                    s_digit = top + 3 - e;
                    s_need = need - before;
                }
                before += v[e];
            }
        }
        // no free place: everything unprotected goes
        if (tid == 0 && need == 0) {
            s_digit = bins - 1;
            s_need = 0;
        }
        cluster_sync();                // the histograms are read everywhere
        prefix |= (uint32_t)s_digit << shift;
        known |= (uint32_t)(bins - 1) << shift;
        need = s_need;
        if (pass < 2)
            for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
    }
    // keys above `prefix` stay, and the first `need` of its equals; a warp's
    // share is contiguous, 32 positions a step
    const int wshare = (share / kSelWarps + 32) / 32 * 32;
    const int w0 = min(c1, c0 + warp * wshare), w1 = min(c1, w0 + wshare);
    auto stays = [&](int s, uint32_t k) -> bool { return s < lo || s >= hi || k > prefix; };
    auto equals = [&](int s, uint32_t k) -> bool { return s >= lo && s < hi && k == prefix; };
    int n_stay = 0, n_eq = 0;
#pragma unroll 4
    for (int s = w0 + lane; s < w1; s += 32) {
        const uint32_t k = key_at(s);
        n_stay += stays(s, k) ? 1 : 0;
        n_eq += equals(s, k) ? 1 : 0;
    }
    n_stay = __reduce_add_sync(0xffffffffu, n_stay);
    n_eq = __reduce_add_sync(0xffffffffu, n_eq);
    if (lane == 0) {
        w_stay[warp] = n_stay;
        w_eq[warp] = n_eq;
    }
    __syncthreads();
    int at = 0, eq_at = 0;             // stays and equals before this warp's share
    {
        int all_stay = 0, all_eq = 0;
        for (int w = 0; w < kSelWarps; ++w) {
            if (w == warp) {
                at = all_stay;
                eq_at = all_eq;
            }
            all_stay += w_stay[w];
            all_eq += w_eq[w];
        }
        if (tid == 0) {
            counts[0] = all_stay;
            counts[1] = all_eq;
        }
    }
    cluster_sync();
    for (int c = 0; c < rank; ++c) {
        at += (int)sm100::ld_cluster_u32(mapa(smem_u32(counts), (uint32_t)c));
        eq_at += (int)sm100::ld_cluster_u32(mapa(smem_u32(counts + 1), (uint32_t)c));
    }
    cluster_sync();                    // no CTA leaves while another reads its counts
    at += min(eq_at, need);
    const unsigned lower = (1u << lane) - 1u;
    for (int s0 = w0; s0 < w1; s0 += 32) {
        const int s = s0 + lane;
        const uint32_t k = s < w1 ? key_at(s) : 0u;
        const bool eq = s < w1 && equals(s, k);
        const unsigned eqs = __ballot_sync(0xffffffffu, eq);
        const bool take = s < w1 && (stays(s, k) || (eq && eq_at + __popc(eqs & lower) < need));
        const unsigned takes = __ballot_sync(0xffffffffu, take);
        if (take) idx[at + __popc(takes & lower)] = s;
        at += __popc(takes);
        eq_at += __popc(eqs);
    }
}

// -------------------------------------------------------------- compaction

constexpr int kMoveThreads = 512;
constexpr int kMoveBuf = 40 * 1024;                  // bytes of a block of rows in a CTA, of two
constexpr int kMoveRows = kMoveBuf / 64;             // most rows of a block
constexpr int kMoveSmem = 2 * kMoveBuf + 3 * kMoveRows * 8;   // two CTAs a SM
constexpr int kMassPer = 16;

// Rows moved in place: row idx[j] of the sequence to row j, j < new_len, as
// idx ascends and idx[j] >= j. A row may be written once all rows up to it are
// read. A cluster takes one slice of the rows' columns (slices do not touch
// each other): a block of rows is read into the shared memory of its CTAs, and
// written after a cluster barrier, while the next block is on its way. grid.x
// counts sequences times the cluster's size, grid.y the slices: of the latent
// rows, then of the key rows, then (4-byte rows, in registers) the weights,
// whose places behind the last kept one become zero.
struct MoveRows {
    uint8_t* rows;
    int bytes, slices;
};

__global__ void __launch_bounds__(kMoveThreads)
cache_compact_kernel(const MoveRows kv, const MoveRows keys, float* __restrict__ mass, int slice, const PagedRows pg,
                     const int* __restrict__ keep_idx, int keep, const int* __restrict__ new_len)
{
    extern __shared__ __align__(16) uint8_t buf[];
    int2* from_to = reinterpret_cast<int2*>(buf + 2 * kMoveBuf);   // [3][kMoveRows] pool rows, x < 0: stays
    const int rank = (int)cluster_ctarank(), size = (int)cluster_size();
    const int b = (int)(blockIdx.x / size), tid = threadIdx.x;
    const int S = pg.max_pages * pg.page_size;
    const int* idx = keep_idx + (size_t)b * keep;
    const int m = max(0, min(min(new_len[b], keep), S));
    int y = (int)blockIdx.y;
    if (y >= kv.slices + keys.slices) {
        float* row = mass + (size_t)b * S;
        const int per = size * kMoveThreads * kMassPer;
        for (int j0 = 0; j0 < m; j0 += per) {
            float v[kMassPer];
            uint32_t moves = 0;
#pragma unroll
            for (int e = 0; e < kMassPer; ++e) {
                const int j = j0 + (rank * kMassPer + e) * kMoveThreads + tid;
                const int s = j < m ? idx[j] : -1;
                v[e] = 0.f;
                if (s > j && s < S) {
                    v[e] = row[s];
                    moves |= 1u << e;
                }
            }
            cluster_sync();
#pragma unroll
            for (int e = 0; e < kMassPer; ++e)
                if ((moves >> e) & 1u) row[j0 + (rank * kMassPer + e) * kMoveThreads + tid] = v[e];
        }
        cluster_sync();
        for (int j = m + rank * kMoveThreads + tid; j < S; j += size * kMoveThreads) row[j] = 0.f;
        return;
    }
    const MoveRows mv = y < kv.slices ? kv : keys;
    if (y >= kv.slices) y -= kv.slices;
    const int col = y * slice, width = min(slice, mv.bytes - col), pieces = width / 16;
    const int rows = min(kMoveRows, kMoveBuf / width);             // of a block, in one CTA
    const int* bt = pg.block_table + (size_t)b * pg.max_pages;
    auto pool_row = [&](int s) -> int {
        const int page = bt[s / pg.page_size];
        return (unsigned)page < (unsigned)pg.num_pages ? page * pg.page_size + s % pg.page_size : -1;
    };
    uint8_t* base = mv.rows + col;
    const int per = size * rows;
    const int blocks = (m + per - 1) / per;
    // where block k's rows of this CTA come from and go
    auto look_up = [&](int k) {
        int2* ft = from_to + (k % 3) * kMoveRows;
        for (int r = tid; r < rows; r += kMoveThreads) {
            const int j = (k * size + rank) * rows + r;
            int2 f = make_int2(-1, -1);
            if (j < m) {
                const int s = idx[j];
                if (s > j && s < S) f = make_int2(pool_row(s), pool_row(j));
                if (f.y < 0) f.x = -1;
            }
            ft[r] = f;
        }
    };
    // this thread's piece of every step-th row
    const int step = kMoveThreads / pieces, r_first = tid / pieces, p = tid - r_first * pieces;
    auto read = [&](int k) {
        const int2* ft = from_to + (k % 3) * kMoveRows;
        const uint32_t dst = smem_u32(buf) + (uint32_t)(k & 1) * kMoveBuf + p * 16;
        if (r_first < step)
            for (int r = r_first; r < rows; r += step)
                if (ft[r].x >= 0)
                    sm100::cp_async16(dst + (uint32_t)(r * width), base + (size_t)ft[r].x * mv.bytes + p * 16, 16);
    };
    if (blocks > 0) look_up(0);
    __syncthreads();
    if (blocks > 0) read(0);
    if (blocks > 1) look_up(1);
    for (int k = 0; k < blocks; ++k) {
        sm100::cp_async_wait_all();
        cluster_sync();                // block k is read everywhere
        if (k + 1 < blocks) read(k + 1);
        if (k + 2 < blocks) look_up(k + 2);
        const int2* ft = from_to + (k % 3) * kMoveRows;
        const uint8_t* src = buf + (k & 1) * kMoveBuf + p * 16;
        if (r_first < step)
            for (int r = r_first; r < rows; r += step)
                if (ft[r].x >= 0)
                    *reinterpret_cast<uint4*>(base + (size_t)ft[r].y * mv.bytes + p * 16) =
                        *reinterpret_cast<const uint4*>(src + r * width);
    }
}

}  // namespace cache_evict
}  // namespace dsa
