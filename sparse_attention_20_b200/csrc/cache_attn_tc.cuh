// Dense MLA attention (MQA mode) of new tokens over the paged latent cache on
// the 5th-generation tensor cores. Row t of sequence b = seq[t] at position
// p = pos[t] sees V(t) = { s <= p }, with a window W > 0 only
// { s <= p : s > p - W or s < sinks }, and
//   x_s = scale q[t,h].c_s,  lse = log sum_V exp x_s,  out = sum_V exp(x_s - lse) c_s[0:512].
//
// A unit is up to 128 (row, head) pairs of consecutive rows of one sequence:
// one row of 128 heads, eight rows of 16. Its keys are read in tiles of 128.
// A cluster of two CTAs runs a unit as one pair MMA (cta_group::2, M = 128):
// each CTA holds 64 of the pairs, so O (64 x 512 fp32, both lane halves of
// 256 TMEM columns), S (64 columns) and two thirds of Q (192 columns) fit its
// tensor memory, and the logits need no exchange. Per tile: S = Q C^T takes 36
// MMAs of N = 128 (each CTA brings 64 of the keys, all 576 columns), O += P
// C[:, 0:512] takes 16 of N = 256 (each CTA brings all 128 keys, its 256
// columns): 32 and 64 clocks each (measured, A in TMEM or shared memory alike), 2176
// a tile, the tensor pipe's rate. Keys cross L2 twice a tile (72 + 64 KB per
// CTA); box loads of 24 to 32 KB reach 85 B/clk/SM from L2 and 7.4 TB/s from
// HBM, single 8 KB ones 22 B/clk, so a tile is loaded in boxes of four slabs of
// 64 columns x 64 keys, through one ring in the order the MMAs consume:
//   Q K(0) K(1) V(0) K(2) V(1) ... K(n-1) V(n-2) Q' K'(0) V(n-1) K'(1) V'(0) ...
// that runs on across units. While the softmax of tile j runs, the tensor pipe
// does PV(j-1) and QK(j+1), of the next unit if need be.
//
// Work is split evenly over the clusters: the units' tiles lie on one line
// (with a constant per unit for its Q and its epilogue) that is cut into equal
// pieces. A unit cut by a boundary leaves fp32 parts that a second kernel
// joins in a fixed order; a cluster leaves at most two.
//
// Keys that some rows of a unit do not see: their logits are replaced by
// -inf whatever the product gave, and where such a key's values hold a NaN or
// an infinity, 0 times which would reach every row, those are zeroed in
// shared memory before PV. A row that does see the key has a logit of NaN or
// +inf, and all of its out is NaN, or (infinite columns that its query meets
// with the opposite sign) one of -inf, and the values' columns that are no
// numbers are NaN in its out, 0 times them, as in tiles that every row sees:
// the O warps write those (spread_non_numbers).
//
// Warps (16 per CTA): 0-7 softmax (two per TMEM lane quarter, 32 of a row's 64
// keys each); 8 loads; 9 MMA issue (even CTA); 10 walks the cluster's piece and
// hands its parts to the others; 12-15 bring a unit's Q into TMEM as soon as
// the last QK of the unit before is done, and take O out and write it, while
// the softmax is at the next unit already. (With Q written by the softmax
// warps behind a unit's last tile a unit of 386 keys took 17000 clocks, so
// 13500; the O warps' 64 KB, 5000 clocks of scattered stores, bound it now.)
#pragma once
#include <cuda.h>

#include <cfloat>

#include "cache_attn.cuh"
#include "sm100.cuh"

namespace dsa {
namespace cache_attn {

using namespace sm100;

constexpr int kRows = 128;                 // (row, head) pairs of a unit
constexpr int kTile = 128;                 // keys of a tile
constexpr int kTcThreads = 512;
constexpr int kPlanWarps = kTcThreads / 32;
constexpr int kSlab = 64 * 128;            // 64 rows x 64 columns bf16, 128B swizzle
constexpr int kSlotBytes = 4 * kSlab;
constexpr int kSlots = 5;
constexpr int kOffQ = 0;                   // columns [384, 576) of Q; the others are in TMEM
constexpr int kOffP = kOffQ + 3 * kSlab;
constexpr int kOffRope = kOffP + 2 * kSlab;
constexpr int kOffRing = kOffRope + 2 * kSlab;
constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
constexpr int kOffRed = kOffBar + 512;                // [2][4][64] row maxima
constexpr int kOffLsum = kOffRed + 2 * 4 * 64 * 4;    // [2][4][64] row sums
constexpr int kOffMax = kOffLsum + 2 * 4 * 64 * 4;    // [2][64] row maxima that the sums refer to
constexpr int kOffBad = kOffMax + 2 * 64 * 4;         // [2][8] flags of the softmax warps
constexpr int kAhead = 4;                             // parts handed out ahead
constexpr int kOffLost = kOffBad + 64;                // [2][8] tiles that they leave to spread_non_numbers
constexpr int kOffParts = kOffLost + 64;              // [kAhead] PartInfo
constexpr int kOffPlan = kOffParts + kAhead * 64;
constexpr int kTcSmem = kOffPlan + 384 + 1024;        // + alignment slack
static_assert(kTcSmem <= 232448, "shared memory");

constexpr uint32_t kColO = 0, kColS = 256, kColQ = 320;

// On the even CTA's barriers: FULL, RFULL (bytes of both CTAs), QT, SFREE, PFULL
// OFREE (arrivals of both). OWN: a slot that the softmax warps look at first
// (the values of a tile that not every row sees whole), QLOAD: a unit's Q, on
// each CTA's own.
enum : int {
    B_FULL = 0, B_EMPTY = 5, B_OWN = 10, B_RFULL = 15, B_REMPTY = 17, B_QT = 19, B_SFULL = 20, B_SFREE = 21,
    B_PFULL = 22, B_PVDONE = 23, B_RED = 24, B_LSUM = 26, B_DRAIN = 28, B_QLOAD = 29,
    B_OFREE = 31, B_PART = 32, B_PARTFREE = 36, B_QFREE = 40, B_COUNT = 41
};

constexpr int kMaxClusters = 74;
// A unit's Q, first softmax and epilogue cost about as much as this many tiles.
constexpr int kUnitCost = 3;
// How many clusters share work `total`: pieces of at least kFullWork, or of
// kMinWork as long as that is no more than kFewParts clusters (one sequence of
// 3000 keys: 20.6 us in six pieces, 24.7 in three; of 30000: 36 us in 59, 32 in
// 32, whose parts the join reads sooner).
constexpr int kMinWork = 4;
constexpr int kFullWork = 8;
constexpr int kFewParts = 32;
__host__ __device__ __forceinline__ long long pieces_of(long long total, int clusters)
{
    const long long few = total / kMinWork < kFewParts ? total / kMinWork : kFewParts;
    const long long n = total / kFullWork > few ? total / kFullWork : few;
    return n < 1 ? 1 : n < clusters ? n : clusters;
}
// Where there are no more units than clusters and the largest is at most this
// much above an even piece (or a full one), each cluster takes a unit whole: a
// second launch and the parts' way through memory cost some 7 us, the time of
// six tiles (64 windows of 1024 keys: 48 us cut evenly, 33 us whole).
constexpr int kWholeSlack = 6;

// The log2 sum of a part in which a row that sees keys has no logit above -inf.
constexpr float kAllLowest = -FLT_MAX;

// A split unit that the cluster of its last tile describes for the join.
struct SplitDesc {
    int t, n_rows;          // first row, (row, head) pairs (0: nothing to join)
    int c_first, c_last;    // clusters that hold its parts
    int start, total;       // its place on the line of work, the line's length
    int ncl, pad;
};

// Workspace: [2 parts per cluster][512 / 4 columns][128 rows][4] fp32 (a warp's
// lanes hold rows), their log2 sums, descriptors.
constexpr size_t kPartBytes = (size_t)kMaxClusters * 2 * kRows * kDv * 4;
constexpr size_t kPartLseBytes = (size_t)kMaxClusters * 2 * kRows * 4;
constexpr size_t kWsBytes = kPartBytes + kPartLseBytes + kMaxClusters * sizeof(SplitDesc);

struct Args {
    PagedRows pg;
    const __nv_bfloat16* kv;
    const int* pos;
    int T, Hq, window, sinks;
};

// What a row of sequence sq at position p sees (false: nothing).
__device__ __forceinline__ bool row_sees(const Args& a, int sq, int p, Visible& v)
{
    v = visible_of((int)min((long long)p + 1, (long long)a.pg.max_pages * a.pg.page_size), p, a.window, a.sinks);
    return sq >= 0 && sq < a.pg.n_seqs && p >= 0;
}

// Rows t .. t + n - 1 of one sequence and the tiles of keys that they see.
struct Unit {
    int t, n, hi, min_hi, max_lo, sink_end;
    int ns, m0, nt;                // sink tiles, first tile after them, tiles in all
    const int* bt;
};

__device__ __forceinline__ int rows_per_unit(int Hq) { return kRows / Hq; }

__device__ __forceinline__ void finish_unit(Unit& u, int lo_min)
{
    u.ns = u.m0 = u.nt = 0;
    if (u.hi < 0) return;
    const int se = min(u.sink_end, u.hi + 1);
    u.ns = (se + kTile - 1) / kTile;
    u.m0 = max(u.ns, lo_min / kTile);
    u.nt = u.ns + max(0, u.hi / kTile - u.m0 + 1);
}

// The unit that starts at row t (lanes = 32: a whole warp takes part; 1: one
// thread). A run of more rows of a sequence is cut every rows_per_unit rows.
template <int lanes>
__device__ __forceinline__ Unit unit_at(const Args& a, int t)
{
    Unit u;
    const int G = rows_per_unit(a.Hq), lane = lanes == 32 ? threadIdx.x & 31 : 0;
    const int sq = a.pg.seq[t];
    int lo_min = INT_MAX;
    u.t = t;
    u.n = 0;
    u.hi = -1;
    u.min_hi = INT_MAX;
    u.max_lo = 0;
    u.sink_end = a.window > 0 ? a.sinks : 0;
    for (int g0 = 0; g0 < G; g0 += lanes) {
        const int r = min(t + g0 + lane, a.T - 1);
        const int sr = a.pg.seq[r], pr = a.pos[r];
        const bool in = g0 + lane < G && t + g0 + lane < a.T && sr == sq;
        int cnt = in ? 1 : 0;
        if (lanes == 32) {
            const unsigned m = __ballot_sync(0xffffffffu, in);
            cnt = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        }
        if (lane < cnt) {
            Visible v;
            if (row_sees(a, sr, pr, v)) {
                u.hi = max(u.hi, v.hi);
                u.min_hi = min(u.min_hi, v.hi);
                u.max_lo = max(u.max_lo, v.lo);
                lo_min = min(lo_min, v.lo);
            } else {
                u.min_hi = -1;
            }
        }
        u.n += cnt;
        if (cnt < lanes) break;
    }
    if (lanes == 32) {
        u.hi = __reduce_max_sync(0xffffffffu, u.hi);
        u.min_hi = __reduce_min_sync(0xffffffffu, u.min_hi);
        u.max_lo = __reduce_max_sync(0xffffffffu, u.max_lo);
        lo_min = __reduce_min_sync(0xffffffffu, lo_min);
    }
    u.bt = a.pg.block_table + (size_t)(u.hi >= 0 ? sq : 0) * a.pg.max_pages;
    finish_unit(u, lo_min);
    return u;
}

// A part as the other warps need it.
struct PartInfo {
    int t, rows;               // first row, (row, head) pairs (without keys: of any number of units)
    int hi, min_hi, max_lo, sink_end;
    int ns, m0;
    int a, nt;                 // first tile and tiles of the part; nt = 0: a unit without keys, -1: no more parts
    int place;                 // its slot among the workspace's parts, -1: the part is the whole unit
    int pad;
    const int* bt;
    long long pad2;
    __device__ __forceinline__ int key0(int j) const { return (a + j < ns ? a + j : m0 + a + j - ns) * kTile; }
    // every row sees keys [s, s + m)
    __device__ __forceinline__ bool all_see(int s, int m) const
    {
        return s + m - 1 <= min_hi && (s >= max_lo || s + m <= sink_end);
    }
};
static_assert(sizeof(PartInfo) == 64, "PartInfo");

// This cluster's piece [w0, w1) of the line of work, and the unit it starts in.
// (The host refuses a line of 2^31 or more; 64-bit divisions here cost a call
// on 200 keys 1 us.)
struct Piece {
    int w0, w1, total, ncl;
    int at, t, parts;       // where the walk goes on behind the first unit, parts handed out so far
    // floor(total c / ncl)
    __device__ __forceinline__ static int begin(int total, int ncl, int c)
    {
        const int q = total / ncl, r = total - q * ncl;
        return c * q + c * r / ncl;
    }
    // the cluster whose piece holds place x
    __device__ __forceinline__ int cluster_of(int x) const
    {
        int c = min(ncl - 1, x / max(1, total / ncl));
        while (begin(total, ncl, c) > x) --c;
        return c;
    }
};

// The piece's share of unit u at place `at`, if any: written to *out, and
// described for the join where the cluster ends a unit that others began.
__device__ __forceinline__ bool part_of(const Args& a, const Piece& pc, int cid, const Unit& u, int at, PartInfo* out,
                                        SplitDesc* desc)
{
    const int d = at + kUnitCost;
    const int b0 = max(0, min(u.nt, pc.w0 - d)), b1 = max(0, min(u.nt, pc.w1 - d));
    if (b0 >= b1 && (u.nt > 0 || at < pc.w0)) return false;
    PartInfo i;
    i.t = u.t;
    i.rows = u.n * a.Hq;
    i.hi = u.hi;
    i.min_hi = u.min_hi;
    i.max_lo = u.max_lo;
    i.sink_end = u.sink_end;
    i.ns = u.ns;
    i.m0 = u.m0;
    i.a = b0;
    i.nt = b1 - b0;
    i.place = b0 > 0 || b1 < u.nt ? cid * 2 + (at < pc.w0 ? 0 : 1) : -1;
    i.pad = 0;
    i.bt = u.bt;
    i.pad2 = 0;
    *out = i;
    if (desc && b1 == u.nt && b0 > 0) {
        SplitDesc s;
        s.t = u.t;
        s.n_rows = i.rows;
        s.c_first = pc.cluster_of(d);
        s.c_last = cid;
        s.start = at;
        s.total = pc.total;
        s.ncl = pc.ncl;
        s.pad = 0;
        *desc = s;
    }
    return true;
}

// Block-wide: finds the units' places on the line of work from seq and pos
// (every CTA does so for itself; a row costs a thread a few loads), and hands
// out the part of the unit that this cluster's piece starts in.
__device__ Piece plan(const Args& a, int cid, int clusters, int* smem, PartInfo* first, SplitDesc* desc,
                      uint32_t first_bar)
{
    int* sums = smem;                   // [16] warp sums
    int* runs = smem + kPlanWarps;      // [16] last run start of each warp's rows
    int* found = smem + 2 * kPlanWarps; // where the walk goes on, parts handed out
    int* units = smem + 3 * kPlanWarps; // [16] units that start in each warp's rows, and their largest
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = rows_per_unit(a.Hq);
    const int per = (a.T + kTcThreads - 1) / kTcThreads;
    const int r0 = min(a.T, tid * per), r1 = min(a.T, r0 + per);
    if (r0 < r1) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.pos + r0));
    auto breaks = [&](int t) { return t == 0 || a.pg.seq[t] != a.pg.seq[t - 1]; };
    // start of the run that row r0 lies in: the last break before or at it (a
    // unit of one row starts anywhere)
    int before = 0;
    if (G > 1) {
        int last = -1;
        for (int t = r0; t < r1; ++t)
            if (breaks(t)) last = t;
        int run = last;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run = max(run, y);
        }
        if (lane == 31) runs[warp] = run;
        __syncthreads();
        before = __shfl_up_sync(0xffffffffu, run, 1);
        if (lane == 0) before = -1;
        for (int w = 0; w < warp; ++w) before = max(before, runs[w]);
    }
    // work of the units that start in this thread's rows
    Unit u;
    int sum = 0, start = before, n_units = 0, largest = 0;
    for (int t = r0; t < r1; ++t) {
        if (G > 1 && breaks(t)) start = t;
        if (G == 1 || (t - start) % G == 0) {
            u = unit_at<1>(a, t);
            sum += u.nt + kUnitCost;
            largest = max(largest, u.nt + kUnitCost);
            ++n_units;
        }
    }
    const int here = n_units;
    if (per == 1) {
        const unsigned m = __ballot_sync(0xffffffffu, here > 0);
        n_units = __popc(m & ((1u << lane) - 1u));
        largest = __reduce_max_sync(0xffffffffu, largest);
        if (lane == 0) {
            units[2 * warp] = __popc(m);
            units[2 * warp + 1] = largest;
        }
    }
    int pre = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += y;
    }
    if (lane == 31) sums[warp] = pre;
    __syncthreads();        // also orders the descriptor's default before a part's
    Piece p;
    p.total = 0;
    pre -= sum;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        if (w < warp) pre += sums[w];
        p.total += sums[w];
    }
    p.ncl = (int)pieces_of(p.total, clusters);
    p.w0 = cid < p.ncl ? Piece::begin(p.total, p.ncl, cid) : p.total;
    p.w1 = cid < p.ncl ? Piece::begin(p.total, p.ncl, cid + 1) : p.total;
    bool mine = p.w0 < p.w1 && sum > 0 && pre <= p.w0 && p.w0 < pre + sum;
    if (per == 1) {
        int all = 0;
        largest = 0;
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) {
            if (w < warp) n_units += units[2 * w];
            all += units[2 * w];
            largest = max(largest, units[2 * w + 1]);
        }
        if (all <= clusters && largest <= max(p.total / p.ncl, kFullWork) + kWholeSlack) {
            // unit cid, whole; its thread alone knows where it lies
            mine = here > 0 && n_units == cid;
            p.w0 = 0;
            p.w1 = cid < all ? p.total : 0;
            if (mine) {
                p.w0 = pre;
                p.w1 = pre + sum;
            }
            p.t = -1;
        } else {
            p.t = 0;
        }
    } else {
        p.t = 0;
    }
    const bool whole = p.t < 0;
    if (mine) {
        int at = pre;
        if (per > 1) {
            start = before;
            for (int t = r0; t < r1; ++t) {
                if (G > 1 && breaks(t)) start = t;
                if (G == 1 || (t - start) % G == 0) {
                    u = unit_at<1>(a, t);
                    if (p.w0 < at + u.nt + kUnitCost) break;
                    at += u.nt + kUnitCost;
                }
            }
        }
        found[0] = at + kUnitCost + u.nt;
        found[1] = u.t + u.n;
        found[2] = part_of(a, p, cid, u, at, first, desc) ? 1 : 0;
        if (found[2]) mbar_arrive(first_bar);
    }
    __syncthreads();
    p.parts = p.w0 < p.w1 ? found[2] : 0;
    p.at = whole ? p.w1 : found[0];     // a whole unit is all of its cluster's work
    p.t = found[1];
    return p;
}

// Waits that last as long as a unit (up to 1.5 s of tiles in 180 GB of cache)
// have this limit; they end with the CTA's abort flag as soon as another gives up.
constexpr uint64_t kUnitWaitNs = 60ull * 1000000000ull;

__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t par, volatile int* abort_flag, int tag, int c,
                                         uint64_t limit_ns = kWaitLimitNs)
{
    return __all_sync(0xffffffffu, mbar_wait<true>(bar, par, abort_flag, tag, c, limit_ns));
}

// Waits on a barrier per lane, all at once (one round costs about as much as a
// wait on one barrier). Bounded; the outcome is the warp's.
__device__ __forceinline__ bool wait_lanes(uint32_t bar, uint32_t par, volatile int* abort_flag, int tag, int c,
                                           uint64_t limit_ns = kWaitLimitNs)
{
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, par))) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        bool mine = mbar_test_wait(bar, par);
        if (__all_sync(0xffffffffu, mine)) return true;
        const bool late = globaltimer_ns() - t0 > limit_ns;
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
            if (late && !mine) report_timeout(tag, c, (int)par);
            *abort_flag = 1;
            return false;
        }
    }
}

// Bits of the 32 keys from s that the row sees.
__device__ __forceinline__ uint32_t seen_bits(const Visible& v, int s)
{
    auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
    return below(v.hi + 1 - s) & (~below(v.lo - s) | below(v.sink_end - s));
}

// Non-finite bf16 halves of w -> 0.
__device__ __forceinline__ uint32_t finite_halves(uint32_t w)
{
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
    return w;
}

// Of a part's nt tiles, tile j stands in this one of 32 groups.
__device__ __forceinline__ int tile_group(int j, int nt) { return (int)((long long)j * 32 / nt); }

// Pair r of a part: NaN in the columns (256 from 256 * side) in which a key that
// its row sees holds no number, for the keys whose values PV read as zeros. The
// row's weight of such a key is 0 or NaN. Rare, so it reads the cache again:
// the tiles of the groups in `where`. To out (orow), or to its place in the
// parts (po).
__device__ __noinline__ void spread_non_numbers(const Args a, const PartInfo p, int r, int side, uint32_t where,
                                                __nv_bfloat16* orow, float4* po)
{
    const int t = p.t + r / a.Hq;
    Visible v;
    if (!row_sees(a, a.pg.seq[t], a.pos[t], v)) return;
#pragma unroll 1
    for (int j = 0; j < p.nt; ++j) {
        const int key0 = p.key0(j);
        if (!((where >> tile_group(j, p.nt)) & 1u) || p.all_see(key0, kTile)) continue;
#pragma unroll 1
        for (int s = key0; s < key0 + kTile; ++s) {
            if (!(seen_bits(v, s) & 1u) || p.all_see(s, 1)) continue;
            const uint4* c = reinterpret_cast<const uint4*>(a.kv + key_row(a.pg, p.bt, 0, s) * kDqk + side * 256);
#pragma unroll 4
            for (int i = 0; i < 32; ++i) {
                const uint4 w4 = __ldg(c + i);
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (((w[e >> 1] >> (16 * (e & 1))) & 0x7F80u) != 0x7F80u) continue;
                    if (po)
                        reinterpret_cast<float*>(po + (size_t)(side * 64 + 2 * i + (e >> 2)) * kRows)[e & 3] =
                            __uint_as_float(0x7FC00000u);
                    else
                        orow[8 * i + e] = __ushort_as_bfloat16((unsigned short)0x7FC0u);
                }
            }
        }
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTcThreads, 1)
mla_attn_paged_tc_kernel(const __grid_constant__ CUtensorMap tm_kv4, const __grid_constant__ CUtensorMap tm_kv1,
                         const __grid_constant__ CUtensorMap tm_q4, const __grid_constant__ CUtensorMap tm_q1,
                         const Args args, float scale_log2,
                         __nv_bfloat16* __restrict__ out, float* __restrict__ lse, float* __restrict__ part_o,
                         float* __restrict__ part_lse, SplitDesc* __restrict__ desc)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t* sgen = smem_raw + (sbase - raw);
    const uint32_t bar0 = sbase + kOffBar;
    uint32_t* taddr_slot = reinterpret_cast<uint32_t*>(sgen + kOffBar + 8 * B_COUNT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sgen + kOffBar + 8 * B_COUNT + 8);
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int cid = (int)(blockIdx.x >> 1), clusters = (int)(gridDim.x >> 1);
    const uint32_t el = elect_one();

    griddep_launch();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(bar(B_FULL + s), 1);
            mbar_init(bar(B_EMPTY + s), 1);
            mbar_init(bar(B_OWN + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(B_RFULL + b), 1);
            mbar_init(bar(B_REMPTY + b), 1);
            mbar_init(bar(B_RED + b), 8);
        }
        // the softmax warps, and those of Q and O, of both CTAs
        mbar_init(bar(B_SFREE), 16);
        mbar_init(bar(B_PFULL), 16);
        mbar_init(bar(B_QT), 8);
        mbar_init(bar(B_OFREE), 8);
        mbar_init(bar(B_QFREE), 1);
        mbar_init(bar(B_SFULL), 1);
        mbar_init(bar(B_PVDONE), 1);
        // of every other unit each: the softmax may be through the next unit (one of a
        // single tile) before the O warps have looked for this one's sums
        mbar_init(bar(B_LSUM), 8);
        mbar_init(bar(B_LSUM + 1), 8);
        mbar_init(bar(B_DRAIN), 1);
        // of every other unit each (a unit's Q may be on its way before the last one's
        // is here): two slots and a rope slot
        mbar_init(bar(B_QLOAD), 3);
        mbar_init(bar(B_QLOAD + 1), 3);
        for (int p = 0; p < kAhead; ++p) {
            mbar_init(bar(B_PART + p), 1);
            mbar_init(bar(B_PARTFREE + p), rank == 0 ? 14 : 13);   // softmax, loads, MMA issue, O
        }
        *abort_flag = 0;
        fence_mbar_init_cluster();
    }
    if (warp == 9) {
        tmem_alloc_pair(smem_u32(taddr_slot), 512);
        tmem_relinquish_pair();
    }
    if (warp == 8 && el) {
        prefetch_tmap(&tm_kv4);
        prefetch_tmap(&tm_kv1);
        prefetch_tmap(&tm_q4);
        prefetch_tmap(&tm_q1);
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();     // the other CTA's barriers exist before any remote arrival
    griddep_wait();
    PartInfo* infos = reinterpret_cast<PartInfo*>(sgen + kOffParts);
    if (rank == 0 && threadIdx.x == 0) desc[cid].n_rows = 0;
    const Piece pc = plan(args, cid, clusters, reinterpret_cast<int*>(sgen + kOffPlan), infos,
                          rank == 0 ? desc + cid : nullptr, bar(B_PART));
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = *taddr_slot;
    // part n of the piece (false: given up); it is handed back at once
    auto take_part = [&](int n, PartInfo& p) -> bool {
        const int at = n % kAhead;
        if (!wait_lanes(bar(B_PART + at), (n / kAhead) & 1, abort_flag, 1050, n)) return false;
        p = infos[at];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PARTFREE + at));
        return true;
    };

    if (warp == 8) {
        // ------------------------------------------------------------ loads
        int slot = 0, rslot = 0, n = 0;
        uint32_t ph = 0, rph = 0;
        bool ok = true;
        const uint32_t full0 = mapa(bar(B_FULL), 0), rfull0 = mapa(bar(B_RFULL), 0);
        // one box of four slabs (columns 64 * z ..) of 64 rows from `row`; with a
        // barrier of this CTA the warps that wait there look at it before the MMA
        // (which counts no bytes then; its arrival comes first, so that whatever
        // follows from the load also follows from the arrival: else the other CTA's
        // bytes for the slot's next turn could fall into this one)
        auto push = [&](const CUtensorMap* tm, int row, int z, uint32_t own) {
            if (!ok) return;
            ok = wait_lanes(bar(B_EMPTY + slot), ph ^ 1u, abort_flag, 1000 + slot, n);
            if (!ok) return;
            if (el) {
                const uint32_t dst = sbase + kOffRing + slot * kSlotBytes;
                if (own) {
                    if (rank == 0) mbar_arrive(bar(B_FULL + slot));
                    mbar_arrive_expect_tx(own, kSlotBytes);
                    tma_load_3d(dst, tm, 0, row, z, own);
                } else {
                    if (rank == 0) mbar_arrive_expect_tx(bar(B_FULL + slot), 2 * kSlotBytes);
                    tma_load_3d_pair(dst, tm, 0, row, z, full0 + 8u * (uint32_t)slot);
                }
            }
            __syncwarp();
            if (++slot == kSlots) {
                slot = 0;
                ph ^= 1u;
            }
        };
        // the last slab (the rope columns)
        auto push_rope = [&](const CUtensorMap* tm, int row, uint32_t own) {
            if (!ok) return;
            ok = wait_lanes(bar(B_REMPTY + rslot), rph ^ 1u, abort_flag, 1010 + rslot, n);
            if (!ok) return;
            if (el) {
                const uint32_t dst = sbase + kOffRope + rslot * kSlab;
                if (own) {
                    if (rank == 0) mbar_arrive(bar(B_RFULL + rslot));
                    mbar_arrive_expect_tx(own, kSlab);
                    tma_load_3d(dst, tm, 0, row, 8, own);
                } else {
                    if (rank == 0) mbar_arrive_expect_tx(bar(B_RFULL + rslot), 2 * kSlab);
                    tma_load_3d_pair(dst, tm, 0, row, 8, rfull0 + 8u * (uint32_t)rslot);
                }
            }
            __syncwarp();
            rslot ^= 1;
            if (rslot == 0) rph ^= 1u;
        };
        PartInfo p;
        int units = 0, pa = 0, pb = 0;   // the last tile's cache rows, its values still to be loaded
        bool pcut = false, before = false;
        const int z = 4 * (int)rank;
        auto push_values = [&]() {
            push(&tm_kv4, pa, z, pcut ? bar(B_OWN + slot) : 0u);
            push(&tm_kv4, pb, z, pcut ? bar(B_OWN + slot) : 0u);
        };
        for (int np = 0; ok; ++np) {
            if (!(ok = take_part(np, p)) || p.nt < 0) break;
            if (p.nt == 0) continue;
            // this CTA's 64 of the unit's pairs (rows behind the last are read as zeros)
            const int qrow = p.t * args.Hq + (int)rank * 64;
            const uint32_t here = bar(B_QLOAD + (units++ & 1));
            push(&tm_q4, qrow, 0, here);
            push(&tm_q4, qrow, 4, here);
            push_rope(&tm_q1, qrow, here);
            // cache rows of the tiles' two blocks of 64 keys, sixteen tiles at a
            // time over the lanes (a block behind the last key reads the one before)
            int rows_l = 0;
            for (int j = 0; j < p.nt && ok; ++j, ++n) {
                if ((j & 15) == 0) {
                    int s = p.key0(min(j + (lane >> 1), p.nt - 1)) + (lane & 1) * 64;
                    if (s > p.hi) s -= 64;
                    rows_l = (int)key_row(args.pg, p.bt, 0, s);
                }
                const int e = (j & 15) * 2;
                const int ra = __shfl_sync(0xffffffffu, rows_l, e), rb = __shfl_sync(0xffffffffu, rows_l, e + 1);
                const int own = rank ? rb : ra;
                push(&tm_kv4, own, 0, 0u);
                push(&tm_kv4, own, 4, 0u);
                push_rope(&tm_kv1, own, 0u);
                if (before) push_values();
                before = true;
                pa = ra;
                pb = rb;
                pcut = !p.all_see(p.key0(j), kTile);
            }
        }
        if (before) push_values();
        if (!ok) {
            // given up: copies in flight land before the CTA gives its shared memory up
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 200000ull) {
            }
        }
    } else if (warp == 9 && rank == 0) {
        // ---------------------------------------------------------- MMA issue
        const uint32_t id_qk = idesc_bf16(128, kTile, false), id_pv = idesc_bf16(128, 256, true);
        const uint64_t d_k = smem_desc(sbase + kOffRing, 16, 1024, kSwizzle128B);
        const uint64_t d_v = smem_desc(sbase + kOffRing, kSlab, 1024, kSwizzle128B);
        const uint64_t d_r = smem_desc(sbase + kOffRope, 16, 1024, kSwizzle128B);
        const uint64_t d_q = smem_desc(sbase + kOffQ, 16, 1024, kSwizzle128B);
        const uint64_t d_p = smem_desc(sbase + kOffP, 16, 1024, kSwizzle128B);
        int slot = 0, rslot = 0, g = 0, n_units = 0, last_nt = 0;
        uint32_t ph = 0, rph = 0;
        bool ok = true;
        // lane 0 waits for the slot, lanes 1 and 2 for other barriers (par > 1: none)
        auto ready = [&](int other, uint32_t par, int tag, int third = 0, uint32_t par3 = 2u) -> bool {
            uint32_t wb = bar(B_FULL + slot), wp = ph;
            if (lane == 1 && par <= 1u) {
                wb = bar(other);
                wp = par;
            }
            if (lane == 2 && par3 <= 1u) {
                wb = bar(third);
                wp = par3;
            }
            return wait_lanes(wb, wp, abort_flag, tag, g);
        };
        auto done = [&]() {
            mma_commit_pair(bar(B_EMPTY + slot), el);
            if (++slot == kSlots) {
                slot = 0;
                ph ^= 1u;
            }
        };
        // S = Q C^T of tile g, once the softmax has read the last S
        auto qk = [&]() -> bool {
            if (!ready(B_SFREE, g > 0 ? (uint32_t)((g - 1) & 1) : 2u, 1220)) return false;
            tc_fence_after();
            uint64_t b = d_k + (uint64_t)(slot * (kSlotBytes >> 4));
#pragma unroll
            for (int kk = 0; kk < 16; ++kk)
                mma_pair_ts(tmem + kColS, tmem + kColQ + kk * 8, b + (kk >> 2) * (kSlab >> 4) + (kk & 3) * 2, id_qk,
                            kk > 0 ? 1u : 0u, el);
            done();
            if (!ready(B_RFULL + rslot, rph, 1230)) return false;
            tc_fence_after();
            b = d_k + (uint64_t)(slot * (kSlotBytes >> 4));
#pragma unroll
            for (int kk = 0; kk < 16; ++kk) {
                const uint64_t bk = b + (kk >> 2) * (kSlab >> 4) + (kk & 3) * 2;
                if (kk < 8)
                    mma_pair_ts(tmem + kColS, tmem + kColQ + (16 + kk) * 8, bk, id_qk, 1u, el);
                else
                    mma_pair_ss(tmem + kColS, d_q + ((kk - 8) >> 2) * (kSlab >> 4) + (kk & 3) * 2, bk, id_qk, 1u, el);
            }
            done();
            b = d_r + (uint64_t)(rslot * (kSlab >> 4));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_pair_ss(tmem + kColS, d_q + 2 * (kSlab >> 4) + kk * 2, b + kk * 2, id_qk, 1u, el);
            mma_commit_pair(bar(B_REMPTY + rslot), el);
            rslot ^= 1;
            if (rslot == 0) rph ^= 1u;
            mma_commit_pair(bar(B_SFULL), el);
            return true;
        };
        // O (+)= P C[:, 0:512] of tile gp of unit `of`, whose first waits until the O of
        // the unit before is read
        auto pv = [&](int gp, bool first, int of) -> bool {
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
                if (!ready(B_PFULL, blk == 0 ? (uint32_t)(gp & 1) : 2u, 1240, B_OFREE,
                           blk == 0 && first && of > 0 ? (uint32_t)((of - 1) & 1) : 2u))
                    return false;
                tc_fence_after();
                const uint64_t b = d_v + (uint64_t)(slot * (kSlotBytes >> 4));
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_pair_ss(tmem + kColO + n * 128, d_p + blk * (kSlab >> 4) + kk * 2,
                                    b + n * (2 * kSlab >> 4) + kk * (16 * 128 >> 4), id_pv,
                                    first && blk == 0 && kk == 0 ? 0u : 1u, el);
                done();
            }
            mma_commit_pair(bar(B_PVDONE), el);
            return true;
        };
        PartInfo p;
        for (int np = 0; ok; ++np) {
            if (!(ok = take_part(np, p)) || p.nt < 0) break;
            if (p.nt == 0) continue;
            ok = wait_lanes(bar(B_QT), n_units & 1, abort_flag, 1250, n_units);
            // Q has been taken out of its two slots and rope slot
            done();
            done();
            mma_commit_pair(bar(B_REMPTY + rslot), el);
            rslot ^= 1;
            if (rslot == 0) rph ^= 1u;
            for (int j = 0; j < p.nt && ok; ++j) {
                ok = qk();
                if (j == p.nt - 1) mma_commit_pair(bar(B_QFREE), el);
                if (ok && g > 0) ok = j > 0 ? pv(g - 1, j == 1, n_units) : pv(g - 1, last_nt == 1, n_units - 1);
                ++g;
            }
            last_nt = p.nt;
            ++n_units;
        }
        if (ok && n_units > 0) ok = pv(g - 1, last_nt == 1, n_units - 1);
        // the last signals of the other CTA
        if (ok && n_units > 0)
            wait_lanes(lane == 0 ? bar(B_SFREE) : bar(B_OFREE), lane == 0 ? (uint32_t)((g - 1) & 1) : (uint32_t)((n_units - 1) & 1),
                       abort_flag, 1260, g);
    } else if (warp == 10) {
        // ------------------------------------------------------------ parts
        int at = pc.at, t = pc.t, np = pc.parts;
        while (true) {
            const bool more = pc.w0 < pc.w1 && at < pc.w1 && t < args.T;
            const int slot = np % kAhead;
            if (!wait_lanes(bar(B_PARTFREE + slot), (uint32_t)(((np / kAhead) & 1) ^ 1), abort_flag, 1060, np,
                            kUnitWaitNs))
                break;
            if (!more) {
                if (el) {
                    infos[slot].nt = -1;
                    mbar_arrive(bar(B_PART + slot));
                }
                break;
            }
            Unit u = unit_at<32>(args, t);
            // units without keys (padding) go as one part, however many follow one
            // another: the softmax warps look for the next part with keys while
            // the O warps wait for the present one, so no more than one part
            // without keys may lie between two with
            while (u.nt == 0 && at >= pc.w0 && at + kUnitCost < pc.w1 && t + u.n < args.T) {
                const Unit v = unit_at<32>(args, t + u.n);
                if (v.nt != 0) break;
                u.n += v.n;
                at += kUnitCost;
            }
            bool mine = false;
            if (el) {
                mine = part_of(args, pc, cid, u, at, infos + slot, rank == 0 ? desc + cid : nullptr);
                if (mine) mbar_arrive(bar(B_PART + slot));
            }
            np += __any_sync(0xffffffffu, mine) ? 1 : 0;
            at += kUnitCost + u.nt;
            t += u.n;
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------- Q in, O out
        // lane i holds pair i % 64 of this CTA's 64: of O columns 0..255 for i < 64,
        // the others for i >= 64
        const int i = (warp & 3) * 32 + lane, side = i >> 6, lr = i & 63;
        const int r = (int)rank * 64 + lr;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const float* lsum_s = reinterpret_cast<const float*>(sgen + kOffLsum);
        const float* max_s = reinterpret_cast<const float*>(sgen + kOffMax);
        const uint32_t ofree0 = mapa(bar(B_OFREE), 0), qt0 = mapa(bar(B_QT), 0);
        const bool wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
        int ring = 0, rope = 0;   // where Q of the next unit lies
        // Q of unit number `units`: columns [0, 384) go to TMEM (row i % 64 in both
        // lanes), the others to their place in shared memory
        auto write_q = [&](int units) -> bool {
            if (!wait_all(bar(B_QLOAD + (units & 1)), (units >> 1) & 1, abort_flag, 1336, units)) return false;
            const uint32_t q0 = sbase + kOffRing + ring % kSlots * kSlotBytes;
            const uint32_t q1 = sbase + kOffRing + (ring + 1) % kSlots * kSlotBytes;
            tc_fence_after();     // the MMAs that read the last Q (QFREE) are over
#pragma unroll 2
            for (int sl = 0; sl < 6; ++sl) {
                const uint32_t src = (sl < 4 ? q0 + sl * kSlab : q1 + (sl - 4) * kSlab) + lr * 128;
                uint32_t w[32];
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    const uint4 x = ld_shared_v4(src + ((v ^ (lr & 7)) << 4));
                    w[4 * v] = x.x; w[4 * v + 1] = x.y; w[4 * v + 2] = x.z; w[4 * v + 3] = x.w;
                }
                tmem_st32(tmem + lane_addr + kColQ + 32 * sl, w);
            }
#pragma unroll 4
            for (int it = 0; it < 12; ++it) {
                const uint32_t o = (uint32_t)(it & 3) * 2048 + i * 16;
                const uint32_t src = it < 8 ? q1 + (2 + (it >> 2)) * kSlab : sbase + kOffRope + (rope & 1) * kSlab;
                st_shared_v4(sbase + kOffQ + (it >> 2) * kSlab + o, ld_shared_v4(src + o));
            }
            tmem_wait_st();
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(qt0);
            return true;
        };
        // the next part with keys; zeros for those without
        int np = 0;
        bool ok = true;
        auto advance = [&](PartInfo& p) -> bool {
            while (true) {
                if (!(ok = take_part(np++, p)) || p.nt < 0) return false;
                if (p.nt > 0) return true;
                for (int rr = r; rr < p.rows; rr += kRows) {
                    const size_t at = (size_t)p.t * args.Hq + rr;
                    uint4* dst = reinterpret_cast<uint4*>(out + at * kDv + side * 256);
                    for (int v = 0; v < 32; ++v) dst[v] = make_uint4(0u, 0u, 0u, 0u);
                    if (side == 0) lse[at] = -INFINITY;
                }
                __syncwarp();
            }
        };
        PartInfo p, pn;
        int uc = 0, g = 0;
        bool have = advance(p);
        if (have) ok = write_q(0);
        while (have && ok) {
            const bool more = advance(pn);
            if (!ok) break;
            // ring places: the values of a unit's last tile lie behind the next unit's
            // Q and first keys (the first unit has none before it)
            ring += 4 * p.nt + (uc > 0 ? 2 : 0);
            rope += 1 + p.nt;
            if (more) {
                if (!wait_all(bar(B_QFREE), uc & 1, abort_flag, 1338, uc, kUnitWaitNs) || !write_q(uc + 1)) break;
            }
            const bool live = r < p.rows;
            const size_t row = (size_t)p.t * args.Hq + r;
            __nv_bfloat16* orow = out + row * kDv + side * 256;
            g += p.nt;
            // row sum over the four threads of the row
            if (!wait_all(bar(B_LSUM + (uc & 1)), (uc >> 1) & 1, abort_flag, 1340, g, kUnitWaitNs)) break;
            const float* ls = lsum_s + (uc & 1) * 256 + lr;
            const float l = (ls[0] + ls[64]) + (ls[128] + ls[192]);
            const float m = max_s[(uc & 1) * 64 + lr];
            float inv = l != 0.f ? 1.f / l : 0.f;
            float lv = l != 0.f ? m + __log2f(l) : -INFINITY;
            if (l == 0.f && live) {
                // no logit above -inf: a row that sees no key gives 0, one that does has no
                // softmax. For the join such a part's sum is the lowest finite number.
                const int t = p.t + r / args.Hq;
                Visible v;
                if (row_sees(args, args.pg.seq[t], args.pos[t], v) && (v.lo <= v.hi || v.sink_end > 0)) {
                    if (p.place >= 0)
                        lv = kAllLowest;
                    else
                        inv = __uint_as_float(0x7FC00000u);
                }
            }
            // tiles with values that PV read as zeros, of rows that see them
            const uint32_t* lost8 = reinterpret_cast<const uint32_t*>(sgen + kOffLost) + (uc & 1) * 8;
            uint32_t where = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) where |= lost8[w];
            if (!wait_all(bar(B_PVDONE), (g - 1) & 1, abort_flag, 1350, g)) break;
            tc_fence_after();
            float4* po = reinterpret_cast<float4*>(part_o) + (size_t)max(p.place, 0) * kRows * (kDv / 4) + r;
#pragma unroll 1
            for (int h0 = 0; h0 < 256; h0 += 64) {
                uint32_t o2[2][32];
                tmem_ld32(tmem + lane_addr + kColO + h0, o2[0]);
                tmem_ld32(tmem + lane_addr + kColO + h0 + 32, o2[1]);
                tmem_wait_ld();
                if (h0 == 192) {
                    // O is in registers (so the signal need not order the loads)
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_relaxed(ofree0);
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const uint32_t (&o)[32] = o2[hh];
                    const int c0 = h0 + 32 * hh;
                if (live && p.place >= 0) {
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        po[(size_t)((side * 256 + c0) / 4 + v) * kRows] =
                            make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                        __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
                } else if (live) {
                    // whole 32-byte sectors where out allows it
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            w[e] = pack_bf16x2(__uint_as_float(o[16 * v + 2 * e]) * inv,
                                               __uint_as_float(o[16 * v + 2 * e + 1]) * inv);
                        if (wide) {
                            st_global_v8(orow + c0 + 16 * v, w);
                        } else {
                            uint4* dst = reinterpret_cast<uint4*>(orow + c0 + 16 * v);
                            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
                }
                __syncwarp();
            }
            if (live && side == 0) {
                if (p.place >= 0)
                    part_lse[(size_t)p.place * kRows + r] = lv;
                else
                    lse[row] = lv * 0.69314718055994531f;
            }
            if (where && live) spread_non_numbers(args, p, r, side, where, orow, p.place >= 0 ? po : nullptr);
            __syncwarp();
            p = pn;
            have = more;
            ++uc;
        }
    } else if (warp < 8) {
        // -------------------------------------------------------- softmax
        // TMEM lane i holds pair i % 64 of this CTA's 64: keys of the tile's first
        // block of 64 for i < 64, of the second for the others; hs halves both
        // once more.
        const int hs = warp >> 2;
        const int i = (warp & 3) * 32 + lane;
        const int side = i >> 6, lr = i & 63;
        const int r = (int)rank * 64 + lr;                  // pair of the unit
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const int grp = side * 2 + hs;
        float* red = reinterpret_cast<float*>(sgen + kOffRed);
        float* lsum_s = reinterpret_cast<float*>(sgen + kOffLsum);
        float* max_s = reinterpret_cast<float*>(sgen + kOffMax);
        int* bad_s = reinterpret_cast<int*>(sgen + kOffBad);
        const uint32_t sfree0 = mapa(bar(B_SFREE), 0), pfull0 = mapa(bar(B_PFULL), 0);
        bool ok = true;
        uint32_t own_ph = 0;      // phase of each slot's OWN
        auto own_slot = [&](int place) -> int {
            const int rs = place % kSlots;
            if (!wait_all(bar(B_OWN + rs), (own_ph >> rs) & 1u, abort_flag, 1330 + rs, place)) return -1;
            own_ph ^= 1u << rs;
            return rs;
        };
        // the next part with keys, and what this thread's pair sees
        int np = 0;
        auto advance = [&](PartInfo& p, Visible& vis) -> bool {
            do {
                if (!take_part(np++, p)) {
                    ok = false;
                    return false;
                }
                if (p.nt < 0) return false;
            } while (p.nt == 0);
            vis.hi = -1;
            vis.lo = vis.sink_end = 0;
            if (r < p.rows) {
                const int t = p.t + r / args.Hq;
                Visible v;
                if (row_sees(args, args.pg.seq[t], args.pos[t], v)) vis = v;
            }
            return true;
        };
        PartInfo u, un;
        Visible vis, vn;
        bool have = advance(u, vis);
        int g = 0, uc = 0;
        int ring = -2;            // ring place of the unit's Q (two less for the first: no values before its K(1))
        while (have && ok) {
            const int nt = u.nt;
            bool more = false;
            float m_use = -INFINITY, l = 0.f;
            uint32_t lost = 0;
            for (int j = 0; j < nt; ++j, ++g) {
                const int key0 = u.key0(j);
                const bool whole = u.all_see(key0, kTile);
                if (!wait_all(bar(B_SFULL), g & 1, abort_flag, 1300, g)) { ok = false; break; }
                tc_fence_after();
                float x[32];
                {
                    uint32_t sr[32];
                    tmem_ld32(tmem + lane_addr + kColS + 32 * hs, sr);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    // the loads' results are here, so the signal need not order them
                    if (lane == 0) mbar_arrive_remote_relaxed(sfree0);
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(sr[e]) * scale_log2;
                }
                if (!whole) {
                    // -inf for a key that the row does not see; a note if the logit of a
                    // key that some row does not see is no number (then neither is
                    // one of its columns: any row tells, in both CTAs alike)
                    const int s0 = key0 + 64 * side + 32 * hs;
                    Visible every;
                    every.lo = u.max_lo;
                    every.hi = u.min_hi;
                    every.sink_end = u.sink_end;
                    const uint32_t bits = seen_bits(vis, s0), all = seen_bits(every, s0);
                    bool bad = false;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        if (!((all >> e) & 1u)) bad |= !(fabsf(x[e]) < INFINITY);
                        if (!((bits >> e) & 1u)) x[e] = -INFINITY;
                    }
                    bad = __any_sync(0xffffffffu, bad);
                    if (bad) {
                        // a row sees such a key with a logit of -inf
                        bool low = false;
#pragma unroll
                        for (int e = 0; e < 32; ++e) low |= ((bits & ~all) >> e & 1u) && x[e] == -INFINITY;
                        if (__any_sync(0xffffffffu, low)) lost |= 1u << tile_group(j, nt);
                    }
                    if (lane == 0) bad_s[(g & 1) * 8 + warp] = bad ? 1 : 0;
                }
                float mx[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) mx[e] = fmaxf(x[e], x[e + 16]);
#pragma unroll
                for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
                    for (int e = 0; e < w; ++e) mx[e] = fmaxf(mx[e], mx[e + w]);
                // row maximum over the four threads that share the row
                float* rd = red + (g & 1) * 256;
                rd[grp * 64 + lr] = mx[0];
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_RED + (g & 1)));
                if (!wait_all(bar(B_RED + (g & 1)), (g >> 1) & 1, abort_flag, 1310, g)) { ok = false; break; }
                const float m_new = fmaxf(m_use, fmaxf(fmaxf(rd[lr], rd[64 + lr]), fmaxf(rd[128 + lr], rd[192 + lr])));
                // the running maximum follows only when it would let P exceed 2^8
                const bool raise = m_new > m_use + 8.f;
                const bool rescale = raise && m_use != -INFINITY;
                const float f = rescale ? ex2(m_use - m_new) : 1.f;
                if (raise) m_use = m_new;
                const float msub = m_use == -INFINITY ? 0.f : m_use;
                // P goes to the MMA in bf16, the type of the values that it meets there: at
                // most half a step, 2^-8 of each weight, like the output's own rounding, and
                // less in a sum over many keys (relative error of out 0.0017 to 0.0022 against
                // 64 bits, 0.0017 of it the output's); its sum is taken before, in fp32
                uint32_t pk[16];
                float ps[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float p0 = ex2(x[2 * e] - msub), p1 = ex2(x[2 * e + 1] - msub);
                    ps[e] = p0 + p1;
                    pk[e] = pack_bf16x2(p0, p1);
                }
#pragma unroll
                for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
                    for (int e = 0; e < w; ++e) ps[e] += ps[e + w];
                l = l * f + ps[0];
                // PV(g-1) has read P and written O
                if (g > 0 && !wait_all(bar(B_PVDONE), (g - 1) & 1, abort_flag, 1320, g)) { ok = false; break; }
                if (__any_sync(0xffffffffu, rescale)) {
                    tc_fence_after();
#pragma unroll 1
                    for (int q4 = 0; q4 < 4; ++q4) {
                        uint32_t o[32];
                        const uint32_t ta = tmem + lane_addr + kColO + 128 * hs + q4 * 32;
                        tmem_ld32(ta, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(ta, o);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    st_shared_v4(sbase + kOffP + side * kSlab + lr * 128 + (((4 * hs + m) ^ (lr & 7)) << 4),
                                 make_uint4(pk[4 * m], pk[4 * m + 1], pk[4 * m + 2], pk[4 * m + 3]));
                if (j == 0) more = advance(un, vn);
                if (!whole) {
                    // ring places of this tile's values: behind the next tile's keys, and
                    // the next unit's Q before those
                    const int v0 = ring + 4 * j + (j < nt - 1 ? 8 : more ? 10 : 6);
                    int bad = 0;
#pragma unroll
                    for (int w = 0; w < 8; ++w) bad |= bad_s[(g & 1) * 8 + w];
#pragma unroll 1
                    for (int blk = 0; blk < 2 && ok; ++blk) {
                        const int rs = own_slot(v0 + blk);
                        ok = rs >= 0;
                        if (!bad || !ok) continue;
                        uint8_t* slab = sgen + kOffRing + rs * kSlotBytes;
#pragma unroll 1
                        for (int rr = (int)threadIdx.x >> 3; rr < 64; rr += 32) {
                            if (u.all_see(key0 + 64 * blk + rr, 1)) continue;
#pragma unroll
                            for (int sl = 0; sl < 4; ++sl) {
                                uint4* v = reinterpret_cast<uint4*>(slab + sl * kSlab + rr * 128) + (threadIdx.x & 7);
                                const uint4 w = *v;
                                *v = make_uint4(finite_halves(w.x), finite_halves(w.y), finite_halves(w.z),
                                                finite_halves(w.w));
                            }
                        }
                    }
                    if (!ok) break;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(pfull0);
            }
            ring += 2 + 4 * nt;
            if (!ok) break;
            // sum and maximum for the warps that take O
            lsum_s[((uc & 1) * 4 + grp) * 64 + lr] = l;
            if (grp == 0) max_s[(uc & 1) * 64 + lr] = m_use;
            if (lane == 0) reinterpret_cast<uint32_t*>(sgen + kOffLost)[(uc & 1) * 8 + warp] = lost;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_LSUM + (uc & 1)));
            u = un;
            vis = vn;
            have = more;
            ++uc;
        }
    }

    if (warp == 9) {
        // every MMA issued, and every signal to either CTA, completes before TMEM
        // and shared memory are given up
        if (rank == 0) mma_commit_pair(bar(B_DRAIN), el);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(bar(B_DRAIN), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_relaxed();   // both CTAs' MMAs, remote arrivals and copies are over
    tc_fence_after();
    if (warp == 9) tmem_dealloc_pair(tmem, 512);
}

// Joins the parts of a split unit, in the order of the clusters:
//   lse = log sum_z 2^lse_z,  out = sum_z 2^(lse_z - lse) o_z.
// CTAs take items of 8 pairs x 256 columns of the units that the clusters'
// descriptors name.
constexpr int kJoinRows = 8;
constexpr int kJoinCols = 256;
constexpr int kJoinThreads = kJoinRows * kJoinCols / 8;       // two groups of four columns a thread
constexpr int kJoinItems = kRows / kJoinRows * (kDv / kJoinCols);   // of a full unit

__global__ void __launch_bounds__(kJoinThreads)
mla_attn_paged_join_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                           const SplitDesc* __restrict__ desc, int clusters, int Hq, __nv_bfloat16* __restrict__ out,
                           float* __restrict__ lse)
{
    __shared__ float wz[kMaxClusters][kJoinRows];
    __shared__ int where[kMaxClusters];
    __shared__ __align__(16) SplitDesc ds[kMaxClusters];
    __shared__ int active[kMaxClusters];       // clusters that ended a split unit
    __shared__ int n_active;
    griddep_launch();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    static_assert(sizeof(SplitDesc) == 32, "two 16-byte pieces");
    for (int i = threadIdx.x; i < 2 * clusters; i += kJoinThreads)
        reinterpret_cast<uint4*>(ds)[i] = reinterpret_cast<const uint4*>(desc)[i];
    __syncthreads();
    if (warp == 0) {
        int n = 0;
        for (int c0 = 0; c0 < clusters; c0 += 32) {
            const bool is = c0 + lane < clusters && ds[c0 + lane].n_rows > 0;
            const unsigned m = __ballot_sync(0xffffffffu, is);
            if (is) active[n + __popc(m & ((1u << lane) - 1u))] = c0 + lane;
            n += __popc(m);
        }
        if (lane == 0) n_active = n;
    }
    __syncthreads();
    for (int item = blockIdx.x; item < n_active * kJoinItems; item += gridDim.x) {
        const SplitDesc d = ds[active[item / kJoinItems]];
        const int e = item % kJoinItems, r0 = e / (kDv / kJoinCols) * kJoinRows, z4 = e % (kDv / kJoinCols);
        if (d.n_rows <= r0) continue;
        const int parts = d.c_last - d.c_first + 1;
        // a thread per row and two groups of four columns; the first parts' values
        // are on their way while the weights are found
        const int rr = threadIdx.x % kJoinRows, c4 = z4 * (kJoinCols / 4) + threadIdx.x / kJoinRows;
        constexpr int kStep = kJoinThreads / kJoinRows, kFirst = 2;
        const float4* p = reinterpret_cast<const float4*>(part_o) + (size_t)c4 * kRows + min(r0 + rr, d.n_rows - 1);
        auto slot_of = [&](int z) -> int {
            const int c = d.c_first + z;
            return c * 2 + (d.start < Piece::begin(d.total, d.ncl, c) ? 0 : 1);
        };
        float4 early[kFirst][2];
#pragma unroll
        for (int z = 0; z < kFirst; ++z) {
            const float4* pz = p + (size_t)slot_of(min(z, parts - 1)) * kRows * (kDv / 4);
            early[z][0] = __ldcs(pz);
            early[z][1] = __ldcs(pz + (size_t)kStep * kRows);
        }
        {
            // a warp per row, lanes over the parts
            const int r = r0 + warp;
            float v[3], m = -INFINITY;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int z = lane + 32 * i;
                v[i] = -INFINITY;
                if (z >= parts) continue;
                const int at = slot_of(z);
                if (warp == 0) where[z] = at;
                if (r < d.n_rows) v[i] = part_lse[at * kRows + r];
                m = fmaxf(m, v[i]);
            }
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float ms = m == -INFINITY ? 0.f : m;
            float l = (exp2f(v[0] - ms) + exp2f(v[1] - ms)) + exp2f(v[2] - ms);
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            // keys seen, and no logit above -inf in any part (nor a NaN): no softmax
            const bool none = m == kAllLowest && l == l;
            const float total = l != 0.f && !none ? ms + log2f(l) : -INFINITY;
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (lane + 32 * i < parts)
                    wz[lane + 32 * i][warp] = none ? __uint_as_float(0x7FC00000u)
                                                   : v[i] == -INFINITY ? 0.f : exp2f(v[i] - total);
            if (lane == 0 && z4 == 0 && r < d.n_rows) lse[(size_t)d.t * Hq + r] = total * 0.69314718055994531f;
        }
        __syncthreads();
        if (r0 + rr < d.n_rows) {
            float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
            auto add = [&](float w, float4 v, float4& a) {
                a.x = fmaf(w, v.x, a.x);
                a.y = fmaf(w, v.y, a.y);
                a.z = fmaf(w, v.z, a.z);
                a.w = fmaf(w, v.w, a.w);
            };
#pragma unroll
            for (int z = 0; z < kFirst; ++z)
                if (z < parts) {
                    add(wz[z][rr], early[z][0], acc[0]);
                    add(wz[z][rr], early[z][1], acc[1]);
                }
#pragma unroll 4
            for (int z = kFirst; z < parts; ++z) {
                const float w = wz[z][rr];
                const float4* pz = p + (size_t)where[z] * kRows * (kDv / 4);
                add(w, __ldcs(pz), acc[0]);
                add(w, __ldcs(pz + (size_t)kStep * kRows), acc[1]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                reinterpret_cast<uint2*>(out + ((size_t)d.t * Hq + r0 + rr) * kDv)[c4 + i * kStep] =
                    make_uint2(pack_bf16x2(acc[i].x, acc[i].y), pack_bf16x2(acc[i].z, acc[i].w));
        }
        __syncthreads();      // the weights make room for the next item's
    }
}
static_assert(kMaxClusters <= 96 && kJoinThreads == 32 * kJoinRows, "the join's lanes and warps");

}  // namespace cache_attn
}  // namespace dsa
