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

constexpr int kSelThreads = 1024;
constexpr int kSelPer = 16;                          // consecutive positions of a thread
constexpr int kSelRound = kSelThreads * kSelPer;     // positions a CTA holds in registers
constexpr int kBins = 2048;
constexpr int kSelSmem = 3 * kBins * 4;

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
    if (warp == 0) {
        int w = warp_sums[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    const int before = warp > 0 ? warp_sums[warp - 1] : 0;
    *total = warp_sums[31];
    __syncthreads();
    return before + x - v;
}

// One cluster per sequence, its positions in contiguous shares over the CTAs
// and threads. The free places (keep - sinks - recent) go to the largest
// weights of the unprotected positions [sinks, n - recent), ties to the lower
// position: a radix select over the order key's bits, 11 + 11 + 10, finds the
// last key that stays and how many of its equals do; each digit's histogram
// is summed over the cluster's shared memory. Up to 16384 positions per CTA
// the weights are read once and stay in registers; longer sequences read them
// again for each digit.
__global__ void __launch_bounds__(kSelThreads)
cache_evict_select_kernel(const float* __restrict__ mass, long long ld, const int* __restrict__ seq_len,
                          int max_len, int keep, int sinks, int recent, int* __restrict__ keep_idx,
                          int* __restrict__ new_len)
{
    extern __shared__ int hist[];      // [3][kBins]
    __shared__ int wsum[32];
    __shared__ int s_digit, s_need;
    __shared__ int counts[2];          // this CTA's positions above the cut (or protected), and equal to it
    const int rank = (int)cluster_ctarank(), size = (int)cluster_size();
    const int b = (int)(blockIdx.x / size), tid = threadIdx.x;
    const int n = max(0, min(seq_len[b], max_len));
    const float* row = mass + b * ld;
    int* idx = keep_idx + (size_t)b * keep;
    if (rank == 0 && tid == 0) new_len[b] = min(n, keep);
    if (n <= keep) {                   // the whole cluster: no barrier is left behind
        for (int j = rank * kSelThreads + tid; j < keep; j += size * kSelThreads) idx[j] = j < n ? j : -1;
        return;
    }
    const int lo = sinks, hi = n - recent;   // unprotected
    // this CTA's share [c0, c1) of the positions, `rounds` times kSelRound of them
    const int share = (int)(((long long)n + (long long)size * kSelPer - 1) / ((long long)size * kSelPer)) * kSelPer;
    const int c0 = min(n, rank * share), c1 = min(n, c0 + share);
    const int rounds = (c1 - c0 + kSelRound - 1) / kSelRound;
    const bool quads = ((reinterpret_cast<uintptr_t>(row) & 15u) == 0);
    uint32_t key[kSelPer];
    auto load = [&](int r) {
        const int s0 = c0 + r * kSelRound + tid * kSelPer;
        if (quads && s0 + kSelPer <= c1) {
#pragma unroll
            for (int e = 0; e < kSelPer; e += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(row + s0 + e));
                key[e] = mass_key(v.x);
                key[e + 1] = mass_key(v.y);
                key[e + 2] = mass_key(v.z);
                key[e + 3] = mass_key(v.w);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kSelPer; ++e) key[e] = s0 + e < c1 ? mass_key(row[s0 + e]) : 0u;
        }
    };
    for (int i = tid; i < 3 * kBins; i += kSelThreads) hist[i] = 0;
    if (rounds == 1) load(0);
    __syncthreads();
    uint32_t prefix = 0, known = 0;          // digits found so far and their bits
    int need = keep - sinks - recent;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
        int* h = hist + pass * kBins;
        for (int r = 0; r < rounds; ++r) {
            if (rounds > 1) load(r);
            const int s0 = c0 + r * kSelRound + tid * kSelPer;
#pragma unroll
            for (int e = 0; e < kSelPer; ++e) {
                const int s = s0 + e;
                if (s >= lo && s < hi && s < c1 && (key[e] & known) == prefix)
                    atomicAdd(&h[(key[e] >> shift) & (bins - 1)], 1);
            }
        }
        cluster_sync();
        // two bins per thread, from the top; their sums over the cluster
        int v[2] = {0, 0};
        const int top = bins - 1 - 2 * tid;
        if (top > 0)
            for (int c = 0; c < size; ++c) {
                const uint32_t at = mapa(smem_u32(h + top - 1), (uint32_t)c);
                v[1] += (int)sm100::ld_cluster_u32(at);
                v[0] += (int)sm100::ld_cluster_u32(at + 4);
            }
        int all;
        const int before = block_scan(v[0] + v[1], wsum, &all);
        if (top > 0 && before < need && before + v[0] + v[1] >= need) {
            const bool first = before + v[0] >= need;
            s_digit = first ? top : top - 1;
            s_need = need - before - (first ? 0 : v[0]);
        }
        // no free place: everything unprotected goes
        if (tid == 0 && need == 0) {
            s_digit = bins - 1;
            s_need = 0;
        }
        __syncthreads();
        prefix |= (uint32_t)s_digit << shift;
        known |= (uint32_t)(bins - 1) << shift;
        need = s_need;
        __syncthreads();
    }
    // keys above `prefix` stay, and the first `need` of its equals
    auto stays = [&](int s, uint32_t k) -> bool { return s < lo || s >= hi || k > prefix; };
    auto equals = [&](int s, uint32_t k) -> bool { return s >= lo && s < hi && k == prefix; };
    int n_stay = 0, n_eq = 0;
    for (int r = 0; r < rounds; ++r) {
        if (rounds > 1) load(r);
        const int s0 = c0 + r * kSelRound + tid * kSelPer;
#pragma unroll
        for (int e = 0; e < kSelPer; ++e)
            if (s0 + e < c1) {
                n_stay += stays(s0 + e, key[e]) ? 1 : 0;
                n_eq += equals(s0 + e, key[e]) ? 1 : 0;
            }
    }
    int cta_stay, cta_eq;
    const int stay_before = block_scan(n_stay, wsum, &cta_stay), eq_before = block_scan(n_eq, wsum, &cta_eq);
    if (tid == 0) {
        counts[0] = cta_stay;
        counts[1] = cta_eq;
    }
    cluster_sync();
    // places taken by the CTAs before this one, and equals among their positions
    int at = 0, eq_at = 0;
    for (int c = 0; c < rank; ++c) {
        at += (int)sm100::ld_cluster_u32(mapa(smem_u32(counts), (uint32_t)c));
        eq_at += (int)sm100::ld_cluster_u32(mapa(smem_u32(counts + 1), (uint32_t)c));
    }
    cluster_sync();                    // no CTA leaves while another reads its counts
    at += min(eq_at, need);
    for (int r = 0; r < rounds; ++r) {
        int st = stay_before, eq = eq_before;
        if (rounds > 1) {
            load(r);
            st = eq = 0;
            const int s0 = c0 + r * kSelRound + tid * kSelPer;
#pragma unroll
            for (int e = 0; e < kSelPer; ++e)
                if (s0 + e < c1) {
                    st += stays(s0 + e, key[e]) ? 1 : 0;
                    eq += equals(s0 + e, key[e]) ? 1 : 0;
                }
            st = block_scan(st, wsum, &cta_stay);
            eq = block_scan(eq, wsum, &cta_eq);
        }
        // equals of this round before this thread's, and the places before it
        int seen = eq_at + eq;
        int place = at + st + min(seen, need) - min(eq_at, need);
        const int s0 = c0 + r * kSelRound + tid * kSelPer;
#pragma unroll
        for (int e = 0; e < kSelPer; ++e) {
            const int s = s0 + e;
            if (s >= c1) continue;
            bool take = stays(s, key[e]);
            if (equals(s, key[e])) take = seen++ < need;
            if (take) idx[place++] = s;
        }
        at += cta_stay + min(eq_at + cta_eq, need) - min(eq_at, need);
        eq_at += cta_eq;
    }
}

// -------------------------------------------------------------- compaction

constexpr int kMoveThreads = 512;
constexpr int kMoveBuf = 48 * 1024;                            // bytes of a block of rows in a CTA, of two
constexpr int kMoveMaxRows = kMoveBuf / 32;                    // a slice is at least 32 bytes wide
constexpr int kMoveSmem = 2 * kMoveBuf + 2 * kMoveMaxRows * 8;
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
    int2* from_to = reinterpret_cast<int2*>(buf + 2 * kMoveBuf);       // [2][kMoveMaxRows] pool rows, x < 0: stays
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
    const int rows = min(kMoveMaxRows, kMoveBuf / width);              // of a block, in one CTA
    const int* bt = pg.block_table + (size_t)b * pg.max_pages;
    auto pool_row = [&](int s) -> int {
        const int page = bt[s / pg.page_size];
        return (unsigned)page < (unsigned)pg.num_pages ? page * pg.page_size + s % pg.page_size : -1;
    };
    uint8_t* base = mv.rows + col;
    // reads block k's rows of this CTA into buffer k & 1
    auto read = [&](int k) {
        int2* ft = from_to + (k & 1) * kMoveMaxRows;
        const int j0 = (k * size + rank) * rows;
        for (int r = tid; r < rows; r += kMoveThreads) {
            const int j = j0 + r;
            int2 f = make_int2(-1, -1);
            if (j < m) {
                const int s = idx[j];
                if (s > j && s < S) f = make_int2(pool_row(s), pool_row(j));
                if (f.y < 0) f.x = -1;
            }
            ft[r] = f;
        }
        __syncthreads();
        const uint32_t dst = smem_u32(buf) + (uint32_t)(k & 1) * kMoveBuf;
        for (int e = tid; e < rows * pieces; e += kMoveThreads) {
            const int r = e / pieces, p = e - r * pieces;
            if (ft[r].x >= 0)
                sm100::cp_async16(dst + (uint32_t)e * 16, base + (size_t)ft[r].x * mv.bytes + p * 16, 16);
        }
    };
    const int per = size * rows;
    const int blocks = (m + per - 1) / per;
    if (blocks > 0) read(0);
    for (int k = 0; k < blocks; ++k) {
        sm100::cp_async_wait_all();
        cluster_sync();                // block k is read everywhere
        if (k + 1 < blocks) read(k + 1);
        const int2* ft = from_to + (k & 1) * kMoveMaxRows;
        const uint4* src = reinterpret_cast<const uint4*>(buf + (k & 1) * kMoveBuf);
        for (int e = tid; e < rows * pieces; e += kMoveThreads) {
            const int r = e / pieces, p = e - r * pieces;
            if (ft[r].x >= 0) *reinterpret_cast<uint4*>(base + (size_t)ft[r].y * mv.bytes + p * 16) = src[e];
        }
    }
}

}  // namespace cache_evict
}  // namespace dsa
