// Eviction from the paged caches by accumulated attention weight: which
// positions of each sequence stay, and the move of their rows to the front.
#pragma once
#include <algorithm>

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

constexpr int kSelThreads = 384;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelHold = 11776;                      // positions a CTA holds in shared memory
constexpr int kSelShare = 16384;                     // positions of a CTA where the cluster can grow
constexpr int kBins = 2048;
constexpr int kSelMaxCluster = 8;
constexpr int kSelSmem = kSelHold * 4 + kBins * 4;

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
// last key that stays and how many of its equals do. Each digit's histogram
// is added up in the first CTA (only the bins in use cross the cluster), which
// names the digit. A CTA keeps the order keys of its first 11776 positions in
// shared memory, so that four CTAs share a SM and 64 sequences of any length
// run at once (with 16384 it is three and two rounds of the card: 46 us
// against 43); the others are read again for each
// pass. Work is bound by instructions, so positions are handled four a lane,
// and protected ones are left out by an order key of 0, which no weight has.
__global__ void __launch_bounds__(kSelThreads, 4)
cache_evict_select_kernel(const float* __restrict__ mass, long long ld, const int* __restrict__ seq_len,
                          int max_len, int keep, int sinks, int recent, int* __restrict__ keep_idx,
                          int* __restrict__ new_len)
{
    extern __shared__ __align__(16) uint32_t sel_smem[];
    uint32_t* held = sel_smem;                                      // [kSelHold] order keys
    int* hist = reinterpret_cast<int*>(sel_smem + kSelHold);       // [kBins]
    __shared__ int wsum[kSelWarps];
    __shared__ int found[2];           // the digit and what is still needed of its bin (first CTA)
    __shared__ int counts[2];          // this CTA's keys above the cut, and equal to it
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
    for (int j = rank * kSelThreads + tid; j < sinks + recent; j += size * kSelThreads)
        idx[j < sinks ? j : keep - recent + j - sinks] = j < sinks ? j : hi + j - sinks;
    // this CTA's share [c0, c0 + 4 groups) of the positions
    const int share = (int)(((long long)n + (long long)size * 4 - 1) / ((long long)size * 4)) * 4;
    const int c0 = min(n, rank * share), c1 = min(n, c0 + share), groups = (c1 - c0 + 3) / 4;
    const int n_held = min(groups, kSelHold / 4);
    const bool quads = (reinterpret_cast<uintptr_t>(row + c0) & 15u) == 0;
    // order keys of positions c0 + 4 g .. + 3, 0 where protected
    auto fetch = [&](int g) -> uint4 {
        const int s = c0 + 4 * g;
        if (quads && s >= lo && s + 4 <= hi) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(row + s));
            return make_uint4(mass_key(v.x), mass_key(v.y), mass_key(v.z), mass_key(v.w));
        }
        auto one = [&](int p) -> uint32_t { return p >= lo && p < hi ? mass_key(row[p]) : 0u; };
        return make_uint4(one(s), one(s + 1), one(s + 2), one(s + 3));
    };
    for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
#pragma unroll 4
    for (int g = tid; g < n_held; g += kSelThreads) *reinterpret_cast<uint4*>(held + 4 * g) = fetch(g);
    auto keys_at = [&](int g) -> uint4 { return g < n_held ? *reinterpret_cast<const uint4*>(held + 4 * g) : fetch(g); };
    cluster_sync();                          // every histogram is zero
    uint32_t prefix = 0, known = 0;          // digits found so far and their bits
    int need = keep - sinks - recent;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
        auto tally = [&](uint32_t k) {
            if ((k & known) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
        };
#pragma unroll 2
        for (int g = tid; g < groups; g += kSelThreads) {
            const uint4 k = keys_at(g);
            tally(k.x);
            tally(k.y);
            tally(k.z);
            tally(k.w);
        }
        __syncthreads();
        if (rank != 0) {
            const uint32_t h0 = mapa(smem_u32(hist), 0);
            for (int i = tid; i < bins; i += kSelThreads) {
                const int v = hist[i];
                if (v) {
                    sm100::red_cluster_add(h0 + 4u * (uint32_t)i, (uint32_t)v);
                    hist[i] = 0;
                }
            }
        }
        cluster_sync();
        if (rank == 0) {
            // bins from the top down, eight per thread
            const int top = bins - 8 - 8 * tid;
            int of[8] = {};
            if (top >= 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    of[e] = hist[top + 7 - e];
                    hist[top + 7 - e] = 0;
                }
            }
            int sum = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += of[e];
            int before = block_scan(sum, wsum);
            if (top >= 0 && before < need && before + sum >= need) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (before < need && before + of[e] >= need) {
                        found[0] = top + 7 - e;
                        found[1] = need - before;
                    }
                    before += of[e];
                }
            }
            // no free place: everything unprotected goes
            if (tid == 0 && need == 0) {
                found[0] = bins - 1;
                found[1] = 0;
            }
        }
        cluster_sync();
        const uint32_t f0 = mapa(smem_u32(found), 0);
        prefix |= sm100::ld_cluster_u32(f0) << shift;
        need = (int)sm100::ld_cluster_u32(f0 + 4);
        known |= (uint32_t)(bins - 1) << shift;
    }
    // keys above `prefix` stay, and the first `need` of its equals; a warp's
    // share is contiguous, 32 groups a step
    const int wshare = (groups / kSelWarps + 32) / 32 * 32;
    const int g0 = min(groups, warp * wshare), g1 = min(groups, g0 + wshare);
    int n_stay = 0, n_eq = 0;
#pragma unroll 4
    for (int g = g0 + lane; g < g1; g += 32) {
        const uint4 k = keys_at(g);
        n_stay += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
        n_eq += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
    }
    n_stay = __reduce_add_sync(0xffffffffu, n_stay);
    n_eq = __reduce_add_sync(0xffffffffu, n_eq);
    if (lane == 0) {
        w_stay[warp] = n_stay;
        w_eq[warp] = n_eq;
    }
    __syncthreads();
    int at = 0, eq_at = 0;             // keys above the cut and equals before this warp's share
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
    cluster_sync();                    // no CTA leaves while another reads its counts or its digit
    at += lo + min(eq_at, need);
    const unsigned lower = (1u << lane) - 1u;
    for (int gg = g0; gg < g1; gg += 32) {
        const int g = gg + lane, s = c0 + 4 * g;
        const uint4 kq = g < g1 ? keys_at(g) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t k[4] = {kq.x, kq.y, kq.z, kq.w};
        unsigned take = 0;             // of this lane's four
#pragma unroll
        for (int e = 0; e < 4; ++e) take |= (k[e] > prefix ? 1u : 0u) << e;
        if (eq_at < need) {            // equals still find a place (the same for the whole warp)
            unsigned eq = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) eq |= (g < g1 && k[e] == prefix ? 1u : 0u) << e;
            if (__any_sync(0xffffffffu, eq != 0)) {
                int before = 0, all = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const unsigned m = __ballot_sync(0xffffffffu, (eq >> e) & 1u);
                    before += __popc(m & lower);
                    all += __popc(m);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if ((eq >> e) & 1u) {
                        if (eq_at + before < need) take |= 1u << e;
                        ++before;
                    }
                eq_at += all;
            }
        }
        int place = at, all = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned m = __ballot_sync(0xffffffffu, (take >> e) & 1u);
            place += __popc(m & lower);
            all += __popc(m);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if ((take >> e) & 1u) idx[place++] = s + e;
        at += all;
    }
}

// -------------------------------------------------------------- compaction

constexpr int kMoveThreads = 512;
constexpr int kMassPer = 16;

// How a compaction is laid out: the width of a slice of columns, the CTAs of a
// cluster, bytes and most rows of a block in a CTA (two are in turn).
struct MoveShape {
    int slice, size, buf, rows;
    size_t smem() const { return 2 * (size_t)buf + 3 * (size_t)rows * 8; }
};

// All CTAs should run at once, with 7.5 MB in flight to fill HBM, and in few
// blocks, each of which costs some 2.5 us of latency. One sequence's 16384 rows
// go in two blocks of 96 KB per CTA, one CTA a SM (14 us; in 40 KB, two a SM, 18);
// 32 sequences' 4099 rows in 48 KB, two CTAs a SM, slices of 192 bytes: 66 us,
// 5.2 TB/s (in 24 KB 86, slices of 384 bytes 95, of 96 bytes 80).
inline MoveShape move_shape(int n_seqs, int kv_bytes, int k_bytes, bool mass, int keep, int sms)
{
    static const int cuts[] = {1, 2, 3, 4, 6, 9, 12, 18};
    MoveShape best = {128, 1, 48 * 1024, 512};
    double best_us = 1e30;
    long long best_total = 0;
    for (int resident = 1; resident <= 2; ++resident)
        for (int n : cuts)
            for (int size = 1; size <= 8; size *= 2) {
                MoveShape m;
                m.slice = ((kv_bytes + n - 1) / n + 31) / 32 * 32;
                m.size = size;
                m.buf = resident == 1 ? 96 * 1024 : 48 * 1024;
                m.rows = resident == 1 ? 1024 : 512;
                if (m.slice < 64 && n > 1) continue;
                const long long total = (long long)n_seqs * size *
                                        (ceil_div(kv_bytes, m.slice) + ceil_div(k_bytes, m.slice) + (mass ? 1 : 0));
                // clusters of 4 and 8 do not fill every group of SMs
                if (total > (long long)resident * (size == 8 ? sms * 13 / 15 : size == 4 ? sms * 14 / 15 : sms)) continue;
                const int rows = std::min(m.rows, m.buf / m.slice);
                const double blocks = ((double)keep / size + rows - 1) / rows;
                const double bytes = 2.0 * n_seqs * keep * (kv_bytes + k_bytes + 4);
                const double us = std::max(2.5 * blocks, bytes / 6e6 / std::min(1.0, total * m.buf / 7.5e6));
                if (us < best_us * 0.99 || (us < best_us * 1.01 && total > best_total)) {
                    best_us = us;
                    best = m;
                    best_total = total;
                }
            }
    return best;
}

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
cache_compact_kernel(const MoveRows kv, const MoveRows keys, float* __restrict__ mass, const MoveShape shape,
                     const PagedRows pg, const int* __restrict__ keep_idx, int keep, const int* __restrict__ new_len)
{
    extern __shared__ __align__(16) uint8_t buf[];
    const int slice = shape.slice, max_rows = shape.rows;
    int2* from_to = reinterpret_cast<int2*>(buf + 2 * shape.buf);  // [3][max_rows] pool rows, x < 0: stays
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
    const int rows = min(max_rows, shape.buf / width);             // of a block, in one CTA
    const int* bt = pg.block_table + (size_t)b * pg.max_pages;
    uint8_t* base = mv.rows + col;
    const int per = size * rows;
    const int blocks = (m + per - 1) / per;
    // Where block k's rows of this CTA come from and go, in three steps that lie
    // an iteration of the loop apart, or the stores of a block, so that no
    // thread waits for its loads: positions, their pages, the table.
    static_assert(kMoveThreads * 2 >= 1024, "rows of a block per thread");
    int pos_of[2];                       // the kept position, -1: none or stays
    int page_from[2], page_to[2], at_from[2], at_to[2];
    auto fetch = [&](int k) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = tid + i * kMoveThreads, j = (k * size + rank) * rows + r;
            const int s = r < rows && j < m ? idx[j] : -1;
            pos_of[i] = s > j && s < S ? s : -1;
        }
    };
    auto find = [&](int k) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (pos_of[i] < 0) continue;
            const int j = (k * size + rank) * rows + tid + i * kMoveThreads;
            const int pf = pos_of[i] / pg.page_size, pt = j / pg.page_size;
            at_from[i] = pos_of[i] - pf * pg.page_size;
            at_to[i] = j - pt * pg.page_size;
            page_from[i] = bt[pf];
            page_to[i] = bt[pt];
        }
    };
    auto note = [&](int k) {
        int2* ft = from_to + (k % 3) * max_rows;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = tid + i * kMoveThreads;
            if (r >= rows) continue;
            int2 f = make_int2(-1, -1);
            if (pos_of[i] >= 0 && (unsigned)page_from[i] < (unsigned)pg.num_pages &&
                (unsigned)page_to[i] < (unsigned)pg.num_pages)
                f = make_int2(page_from[i] * pg.page_size + at_from[i], page_to[i] * pg.page_size + at_to[i]);
            ft[r] = f;
        }
    };
    auto look_up = [&](int k) {
        fetch(k);
        find(k);
        note(k);
    };
    // this thread's piece of every step-th row
    const int step = kMoveThreads / pieces, r_first = tid / pieces, p = tid - r_first * pieces;
    auto read = [&](int k) {
        const int2* ft = from_to + (k % 3) * max_rows;
        const uint32_t dst = smem_u32(buf) + (uint32_t)(k & 1) * (uint32_t)shape.buf + p * 16;
        if (r_first < step)
            for (int r = r_first; r < rows; r += step)
                if (ft[r].x >= 0)
                    sm100::cp_async16(dst + (uint32_t)(r * width), base + (size_t)ft[r].x * mv.bytes + p * 16, 16);
    };
    if (blocks > 0) look_up(0);
    __syncthreads();
    if (blocks > 0) read(0);
    if (blocks > 1) look_up(1);
    if (blocks > 2) fetch(2);
    for (int k = 0; k < blocks; ++k) {
        // block k is read everywhere: its copies have landed, so the barrier need
        // not order anything (a release waits for the last block's stores)
        sm100::cp_async_wait_all();
        __syncthreads();
        if (size > 1) sm100::cluster_sync_relaxed();
        if (k + 1 < blocks) read(k + 1);
        if (k + 2 < blocks) find(k + 2);
        const int2* ft = from_to + (k % 3) * max_rows;
        const uint8_t* src = buf + (k & 1) * shape.buf + p * 16;
        if (r_first < step)
            for (int r = r_first; r < rows; r += step)
                if (ft[r].x >= 0)
                    *reinterpret_cast<uint4*>(base + (size_t)ft[r].y * mv.bytes + p * 16) =
                        *reinterpret_cast<const uint4*>(src + r * width);
        if (k + 2 < blocks) note(k + 2);
        if (k + 3 < blocks) fetch(k + 3);
    }
}

}  // namespace cache_evict
}  // namespace dsa
