// The attention weight that each cached token receives (tensor cores):
//   mass[b,s] += sum over the rows t of sequence b that see s, and heads h, of
//                exp(x_{t,h,s} - lse[t,h]),  x = scale q[t,h].c_s.
//
// Keys are the M side (S^T = C Q^T), so that a key's sum over rows and heads
// runs along one TMEM lane and needs no exchange between threads. A cluster of
// two CTAs does a tile of 256 keys (pair MMA, M = 256: 128 keys per CTA) against
// 256 (row, head) pairs at a time (N = 256, each CTA brings half of them; N =
// 128 where a step has no more). The tile's keys stay in shared memory (9 slabs
// of 64 columns, 144 KB) for all of the sequence's rows, Q streams through a
// ring of 16 KB slots: 32 B per clock and SM from L2 at the tensor pipe's rate.
// With one row per sequence a slab of keys is free as soon as its MMAs are done
// and the next tile's is on its way: 144 KB in flight per SM, bound by HBM.
//
// The (tile, 256 pairs) steps of all sequences lie on one line that the
// clusters share evenly; a tile cut by a boundary leaves partial sums that a
// second kernel adds in order, so results do not depend on timing. Steps none
// of whose rows sees a key of the tile are passed over.
//
// Warps (11 per CTA): 0-7 sums (two per TMEM lane quarter, half of the columns
// each), 8 loads, 9 MMA issue (even CTA), 10 the steps: it walks the piece and
// hands each step, with its columns' lse and keys seen, to the others up to
// four steps ahead. (Each warp walking for itself put 1400 to 1900 clocks of
// load latency between two steps' MMAs, and the columns' loads 4000 between
// two steps' sums: 256 rows over 12K keys took 505 us.)
#pragma once
#include <cuda.h>

#include "cache_attn_tc.cuh"
#include "sm100.cuh"

namespace dsa {
namespace cache_mass {

using namespace sm100;
using cache_attn::Args;
using cache_attn::Visible;
using cache_attn::visible_of;
using cache_attn::wait_all;
using cache_attn::wait_lanes;

constexpr int kDqk = cache_attn::kDqk;
constexpr int kSlabs = kDqk / 64;
constexpr int kTile = 256;                 // keys of a tile (both CTAs)
constexpr int kPairs = 256;                // (row, head) pairs of a step
constexpr int kThreads = 352;
constexpr int kKSlab = 128 * 128;          // 128 keys x 64 columns
constexpr int kQSlot = 128 * 128;          // 128 pairs x 64 columns
constexpr int kQSlots = 4;
constexpr int kOffK = 0;
constexpr int kOffQ = kOffK + kSlabs * kKSlab;
constexpr int kOffBar = kOffQ + kQSlots * kQSlot;
constexpr int kAhead = 4;                                 // steps handed out ahead
constexpr int kOffCol = kOffBar + 512;                    // [kAhead][256] lse2, last and first key seen
constexpr int kOffHalf = kOffCol + kAhead * 3 * kPairs * 4;   // [kAhead][128] sums of the second column half
constexpr int kOffStep = kOffHalf + kAhead * 128 * 4;          // [kAhead] StepInfo
// Up to this many sequences every CTA makes the plan itself, in its shared
// memory; a kernel before it takes 5 us and the time between two launches.
constexpr int kNearSeqs = 64;
constexpr int kOffHead = kOffStep + kAhead * 64;
constexpr int kOffSeqs = kOffHead + 320;
constexpr int kSmem = kOffSeqs + kNearSeqs * 32 + 1024;
enum : int {
    B_KFULL = 0, B_KEMPTY = 9, B_QFULL = 18, B_QEMPTY = 22, B_DFULL = 26, B_DFREE = 28, B_STEP = 30,
    B_STEPFREE = 34, B_HALF = 38, B_DRAIN = 42, B_COUNT = 43
};

constexpr int kMaxClusters = cache_attn::kMaxClusters;
constexpr int kTileCost = 1;     // of a tile's keys and epilogue, in steps
// Least work of a cluster: one tile and step. (Four sequences of 2000 keys, one
// token each: 12.5 us, with a least work of 6 20.4.)
constexpr int kMinWork = 2;

// What the plan kernel writes: rows and keys of a sequence, and where its
// tiles start on the line of work.
struct SeqPlan {
    int t_min, t_max;       // its rows lie in [t_min, t_max]
    int hi, lo;             // keys that they see lie in [lo, hi] and [0, sink_end)
    long long start;
    long long pad;
};
struct Header {
    long long total;
    int ncl, pad;
    int first[kMaxClusters];      // sequence in which a cluster's piece starts
};
// A tile whose partial sums cluster c_last's descriptor names.
struct SplitTile {
    int b, tile;                 // b < 0: none
    int c_first, c_last;
    long long base, total;
    int ncl, pad;
};

static_assert(kSmem <= 232448, "shared memory");

constexpr size_t kHeaderBytes = 512;
constexpr size_t kDescBytes = kMaxClusters * sizeof(SplitTile);
constexpr size_t kPartBytes = (size_t)kMaxClusters * 2 * kTile * 4;
static_assert(sizeof(Header) <= 320 && sizeof(SeqPlan) == 32 && 320 <= kHeaderBytes, "header");
constexpr size_t kFixedBytes = (kHeaderBytes + kDescBytes + kPartBytes + 255) / 256 * 256;

__host__ __device__ __forceinline__ size_t ws_bytes(int n_seqs) { return kFixedBytes + (size_t)n_seqs * sizeof(SeqPlan); }

struct Ws {
    Header* head;
    SplitTile* desc;
    float* parts;
    SeqPlan* seqs;
};

__host__ __device__ __forceinline__ Ws ws_of(void* p)
{
    uint8_t* b = reinterpret_cast<uint8_t*>(p);
    Ws w;
    w.head = reinterpret_cast<Header*>(b);
    w.desc = reinterpret_cast<SplitTile*>(b + kHeaderBytes);
    w.parts = reinterpret_cast<float*>(b + kHeaderBytes + kDescBytes);
    w.seqs = reinterpret_cast<SeqPlan*>(b + kFixedBytes);
    return w;
}

// Tiles of a sequence: those of the first tokens, then from lo on.
struct Tiles {
    int ns, m0, nt;
    __device__ __forceinline__ int key0(int i) const { return (i < ns ? i : m0 + i - ns) * kTile; }
};

__device__ __forceinline__ Tiles tiles_of(int lo, int hi, int sink_end)
{
    Tiles r;
    r.ns = r.m0 = r.nt = 0;
    if (hi < 0) return r;
    r.ns = (min(sink_end, hi + 1) + kTile - 1) / kTile;
    r.m0 = max(r.ns, lo / kTile);
    r.nt = r.ns + max(0, hi / kTile - r.m0 + 1);
    return r;
}

__device__ __forceinline__ int rows_per_step(int Hq) { return kPairs / Hq; }
__device__ __forceinline__ int steps_of(const SeqPlan& s, int Hq)
{
    return s.t_max < s.t_min ? 0 : (s.t_max - s.t_min) / rows_per_step(Hq) + 1;
}
__device__ __forceinline__ long long piece_begin(long long total, int ncl, int c) { return total * c / ncl; }

constexpr int kPlanThreads = 1024;
constexpr int kPlanSeqs = 1024;     // sequences that the plan kernel handles in shared memory

// A block of `threads` threads: rows and keys of each sequence, then the line
// of work, into w.head and w.seqs; seqs is where it works (w.seqs or shared
// memory), wsum a shared word pair per warp.
template <int threads>
__device__ void plan_block(const Args& a, int clusters, const Ws& w, volatile SeqPlan* seqs, long long* wsum)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int b = tid; b < a.pg.n_seqs; b += threads) {
        seqs[b].t_min = seqs[b].lo = INT_MAX;
        seqs[b].t_max = seqs[b].hi = -1;
    }
    __syncthreads();
    const int sink_end = a.window > 0 ? a.sinks : 0;
    for (int t0 = 0; t0 < a.T; t0 += threads) {
        const int t = t0 + tid;
        int b = -1, hi = -1, lo = INT_MAX;
        if (t < a.T) {
            Visible v;
            const int sq = a.pg.seq[t];
            if (cache_attn::row_sees(a, sq, a.pos[t], v)) {
                b = sq;
                hi = v.hi;
                lo = v.lo;
            }
        }
        int same = 0;
        __match_all_sync(0xffffffffu, b, &same);
        int t_min = t, t_max = t;
        bool mine = b >= 0;
        if (same) {
            t_min = __reduce_min_sync(0xffffffffu, t);
            t_max = __reduce_max_sync(0xffffffffu, t);
            hi = __reduce_max_sync(0xffffffffu, hi);
            lo = __reduce_min_sync(0xffffffffu, lo);
            mine = mine && lane == 0;
        }
        if (mine) {
            atomicMin(const_cast<int*>(&seqs[b].t_min), t_min);
            atomicMax(const_cast<int*>(&seqs[b].t_max), t_max);
            atomicMax(const_cast<int*>(&seqs[b].hi), hi);
            atomicMin(const_cast<int*>(&seqs[b].lo), lo);
        }
    }
    __syncthreads();
    const int per = ceil_div(a.pg.n_seqs, threads);
    const int b0 = min(a.pg.n_seqs, tid * per), b1 = min(a.pg.n_seqs, b0 + per);
    auto cost = [&](int b) -> long long {
        SeqPlan s;
        s.t_min = seqs[b].t_min;
        s.t_max = seqs[b].t_max;
        const Tiles k = tiles_of(seqs[b].lo, seqs[b].hi, sink_end);
        return (long long)k.nt * (steps_of(s, a.Hq) + kTileCost);
    };
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += cost(b);
    long long pre = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += y;
    }
    if (lane == 31) wsum[warp] = pre;
    __syncthreads();
    long long base = 0, total = 0;
#pragma unroll
    for (int i = 0; i < threads / 32; ++i) {
        if (i < warp) base += wsum[i];
        total += wsum[i];
    }
    pre += base - sum;
    const int ncl = total == 0 ? 0 : (int)max(1ll, min((long long)clusters, total / kMinWork));
    if (tid == 0) {
        w.head->total = total;
        w.head->ncl = ncl;
    }
    for (int b = b0; b < b1; ++b) {
        const long long c = cost(b);
        if (seqs != w.seqs) {
            SeqPlan s;
            s.t_min = seqs[b].t_min;
            s.t_max = seqs[b].t_max;
            s.hi = seqs[b].hi;
            s.lo = seqs[b].lo;
            s.start = pre;
            s.pad = 0;
            w.seqs[b] = s;
        }
        seqs[b].start = pre;
        pre += c;
    }
    __syncthreads();
    // the sequence in which each cluster's piece starts: the last one that starts
    // no later (those without work start where the next one does)
    if (tid < ncl) {
        const long long w0 = piece_begin(total, ncl, tid);
        int l = 0, r = a.pg.n_seqs - 1;
        while (l < r) {
            const int m = (l + r + 1) / 2;
            if (seqs[m].start <= w0)
                l = m;
            else
                r = m - 1;
        }
        w.head->first[tid] = l;
    }
}

// For more sequences than each CTA of the main kernel plans for itself.
__global__ void __launch_bounds__(kPlanThreads)
cache_mass_plan_kernel(const Args a, int clusters, void* ws)
{
    __shared__ long long wsum[32];
    __shared__ SeqPlan near[kPlanSeqs];
    griddep_launch();
    griddep_wait();
    const Ws w = ws_of(ws);
    plan_block<kPlanThreads>(a, clusters, w, a.pg.n_seqs <= kPlanSeqs ? near : w.seqs, wsum);
}

// What row t sees if it belongs to sequence b (false: nothing).
__device__ __forceinline__ bool sees(const Args& a, int b, int t, Visible& v)
{
    const int sq = a.pg.seq[t], p = a.pos[t];
    v = visible_of((int)min((long long)p + 1, (long long)a.pg.max_pages * a.pg.page_size), p, a.window, a.sinks);
    return sq == b && p >= 0;
}

// Rows [t0, t0 + n) as a step of sequence b (a whole warp takes part): what
// those of them that belong to b see.
struct StepRange {
    int hi, min_hi, lo, max_lo;
};

__device__ __forceinline__ StepRange step_range(const Args& a, int b, int t0, int n)
{
    StepRange r;
    r.hi = -1;
    r.min_hi = r.lo = INT_MAX;
    r.max_lo = 0;
    for (int i = threadIdx.x & 31; i < n; i += 32) {
        Visible v;
        if (sees(a, b, t0 + i, v)) {
            r.hi = max(r.hi, v.hi);
            r.min_hi = min(r.min_hi, v.hi);
            r.lo = min(r.lo, v.lo);
            r.max_lo = max(r.max_lo, v.lo);
        }
    }
    r.hi = __reduce_max_sync(0xffffffffu, r.hi);
    r.min_hi = __reduce_min_sync(0xffffffffu, r.min_hi);
    r.lo = __reduce_min_sync(0xffffffffu, r.lo);
    r.max_lo = __reduce_max_sync(0xffffffffu, r.max_lo);
    return r;
}

// One step of a cluster's piece.
struct Step {
    int b, tile, key0, hi_b;   // sequence, its tile, the tile's first key, the last key any of its rows sees
    int t0, n;                 // rows; n = 0: no row of this share sees the tile (partial sums of zero are due)
    StepRange rg;
    bool split;
    long long base;            // the tile's place on the line of work
};

// What the other warps need to know of a step.
struct StepInfo {
    int N;          // columns; 0: no step, only a share's end; -1: no more
    int whole;      // every column sees each of this CTA's 128 keys
    int seen;       // some column sees one of them
    int last;       // the last step of this cluster's share of the tile
    int fresh;      // its first one
    int b, key0;
    int part;       // where its partial sums go, -1: the share is the whole tile
    int qrow;       // first (row, head) pair
    int row[2];     // cache rows of this CTA's two blocks of 64 keys
    int pad[5];
};
static_assert(sizeof(StepInfo) == 64, "StepInfo");

// What a look for the next step finds. The waits of the warps that take the steps
// have a limit, so a walk that passes over many (a sequence with few rows far
// apart among others', sequences without rows) says so now and then.
enum : int { kNoMore = 0, kFound = 1, kStillLooking = 2 };
constexpr int kLookMost = 4096;      // steps and sequences passed over in one go: some 10 ms at most

struct StepWalk {
    long long w0, w1, total, base;
    int ncl, b, tile, q, q1, nq;
    bool loaded, in_tile, any;
    SeqPlan s;
    Tiles k;
    // sequence b (false: it has no tiles)
    __device__ __forceinline__ bool load(const Args& a, const Ws& w)
    {
        s = w.seqs[b];
        k = tiles_of(s.lo, s.hi, a.window > 0 ? a.sinks : 0);
        nq = steps_of(s, a.Hq);
        return k.nt > 0;
    }
    __device__ __forceinline__ StepWalk(const Args& a, const Ws& w, int cid)
    {
        total = w.head->total;
        ncl = w.head->ncl;
        loaded = in_tile = any = false;
        b = a.pg.n_seqs;
        w0 = w1 = base = 0;
        tile = q = q1 = nq = 0;
        if (cid >= ncl) return;
        w0 = piece_begin(total, ncl, cid);
        w1 = piece_begin(total, ncl, cid + 1);
        b = w.head->first[cid];
        loaded = load(a, w);      // a cluster's first sequence has tiles
        tile = (int)((w0 - s.start) / (nq + kTileCost));
        base = s.start + (long long)tile * (nq + kTileCost);
    }
    __device__ __forceinline__ int next(const Args& a, const Ws& w, Step& st)
    {
        int passed = 0;
        while (b < a.pg.n_seqs && base < w1) {
            if (!loaded) {
                loaded = load(a, w);
                if (!loaded) {
                    ++b;
                    if (++passed == kLookMost) return kStillLooking;
                    continue;
                }
            }
            const long long d = base + kTileCost;
            if (!in_tile) {
                q = (int)max(0ll, min((long long)nq, w0 - d));
                q1 = (int)max(0ll, min((long long)nq, w1 - d));
                in_tile = true;
                any = false;
                st.split = q < q1 && (q > 0 || q1 < nq);
            } else {
                const int qa = (int)max(0ll, min((long long)nq, w0 - d));
                st.split = qa > 0 || q1 < nq;
            }
            st.b = b;
            st.tile = tile;
            st.key0 = k.key0(tile);
            st.hi_b = s.hi;
            st.base = base;
            const int G = rows_per_step(a.Hq), sink_end = a.window > 0 ? a.sinks : 0;
            while (q < q1) {
                st.t0 = s.t_min + q * G;
                st.n = min(G, s.t_max + 1 - st.t0);
                st.rg = step_range(a, b, st.t0, st.n);
                ++q;
                if (st.key0 <= st.rg.hi && (st.key0 + kTile > st.rg.lo || st.key0 < sink_end)) {
                    any = true;
                    return kFound;
                }
                if (++passed == kLookMost) return kStillLooking;
            }
            // the tile's share is over
            in_tile = false;
            const bool due = st.split && !any;
            base += nq + kTileCost;
            if (++tile == k.nt) {
                ++b;
                tile = 0;
                loaded = false;
            }
            if (due) {
                st.n = 0;
                return kFound;
            }
        }
        return kNoMore;
    }
};

// Limit of the waits that the other CTA's share of a step is part of: each CTA
// walks for itself, so after a long look they may be seconds apart.
constexpr uint64_t kApartNs = cache_attn::kUnitWaitNs;

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
cache_mass_tc_kernel(const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_q128,
                     const __grid_constant__ CUtensorMap tm_q64, const float* __restrict__ lse, const Args args,
                     float scale_log2, void* ws_raw, float* __restrict__ mass)
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
    const int cid = (int)(blockIdx.x >> 1);

    griddep_launch();
    if (threadIdx.x == 0) {
        for (int k = 0; k < kSlabs; ++k) {
            mbar_init(bar(B_KFULL + k), 1);
            mbar_init(bar(B_KEMPTY + k), 1);
        }
        for (int s = 0; s < kQSlots; ++s) {
            mbar_init(bar(B_QFULL + s), 1);
            mbar_init(bar(B_QEMPTY + s), 1);
        }
        for (int d = 0; d < 2; ++d) {
            mbar_init(bar(B_DFULL + d), 1);
            mbar_init(bar(B_DFREE + d), 16);    // the summing warps of both CTAs
        }
        for (int d = 0; d < kAhead; ++d) {
            mbar_init(bar(B_STEP + d), 1);
            mbar_init(bar(B_HALF + d), 4);
            mbar_init(bar(B_STEPFREE + d), rank == 0 ? 10 : 9);   // sums, loads, MMA issue
        }
        mbar_init(bar(B_DRAIN), 1);
        *abort_flag = 0;
        fence_mbar_init_cluster();
    }
    if (warp == 9) {
        tmem_alloc_pair(smem_u32(taddr_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the other CTA's barriers exist before any remote arrival
    tc_fence_after();
    griddep_wait();
    const uint32_t tmem = *taddr_slot;
    const uint32_t el = elect_one();
    Ws ws = ws_of(ws_raw);
    if (args.pg.n_seqs <= kNearSeqs) {
        ws.head = reinterpret_cast<Header*>(sgen + kOffHead);
        ws.seqs = reinterpret_cast<SeqPlan*>(sgen + kOffSeqs);
        plan_block<kThreads>(args, (int)(gridDim.x >> 1), ws, ws.seqs,
                             reinterpret_cast<long long*>(sgen + kOffBar + 384));
    }
    if (rank == 0 && threadIdx.x == 0) ws.desc[cid].b = -1;
    __syncthreads();
    bool issued_any = false;
    // pairs of a step as the MMA's N
    auto n_of = [&](const Step& s) -> int { return s.n * args.Hq > 128 ? 256 : 128; };
    // step gd for the loads' and the issuing warp, which need nothing more of it
    auto take_step = [&](int gd, StepInfo& st) -> bool {
        const int at = gd % kAhead;
        if (!wait_lanes(bar(B_STEP + at), (gd / kAhead) & 1, abort_flag, 2050, gd, kApartNs)) return false;
        st = reinterpret_cast<const StepInfo*>(sgen + kOffStep)[at];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_STEPFREE + at));
        return true;
    };

    if (warp == 8) {
        // ------------------------------------------------------------ loads
        if (el) {
            prefetch_tmap(&tm_kv);
            prefetch_tmap(&tm_q128);
            prefetch_tmap(&tm_q64);
        }
        const uint32_t kfull0 = mapa(bar(B_KFULL), 0), qfull0 = mapa(bar(B_QFULL), 0);
        int slot = 0, n_tiles = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int gd = 0; ok; ++gd) {
            StepInfo st;
            if (!(ok = take_step(gd, st))) break;
            if (st.N < 0) break;
            if (st.N == 0) continue;
            const bool fresh = st.fresh != 0;
            const int N = st.N;
            const int qrow = st.qrow + (int)rank * (N / 2);
            for (int k = 0; k < kSlabs; ++k) {
                // a fresh tile waits for its slab of keys, too
                const bool two = fresh && lane == 1;
                ok = wait_lanes(two ? bar(B_KEMPTY + k) : bar(B_QEMPTY + slot), two ? (uint32_t)((n_tiles & 1) ^ 1) : ph ^ 1u,
                                abort_flag, 2000 + k, n_tiles, kApartNs);
                if (!ok) break;
                if (el) {
                    if (fresh) {
                        if (rank == 0) mbar_arrive_expect_tx(bar(B_KFULL + k), 2 * kKSlab);
                        const uint32_t dst = sbase + kOffK + k * kKSlab;
                        tma_load_3d_pair(dst, &tm_kv, 0, st.row[0], k, kfull0 + 8u * (uint32_t)k);
                        tma_load_3d_pair(dst + kKSlab / 2, &tm_kv, 0, st.row[1], k, kfull0 + 8u * (uint32_t)k);
                    }
                    if (rank == 0) mbar_arrive_expect_tx(bar(B_QFULL + slot), (uint32_t)N * 128u);
                    tma_load_3d_pair(sbase + kOffQ + slot * kQSlot, N == 256 ? &tm_q128 : &tm_q64, 0, qrow, k,
                                     qfull0 + 8u * (uint32_t)slot);
                }
                __syncwarp();
                if (++slot == kQSlots) {
                    slot = 0;
                    ph ^= 1u;
                }
            }
            if (fresh) ++n_tiles;
        }
        if (!ok) {
            // given up: copies in flight land before the CTA gives its shared memory up
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 200000ull) {
            }
        }
    } else if (warp == 9 && rank == 0) {
        // ---------------------------------------------------------- MMA issue
        const uint64_t d_k = smem_desc(sbase + kOffK, 16, 1024, kSwizzle128B);
        const uint64_t d_q = smem_desc(sbase + kOffQ, 16, 1024, kSwizzle128B);
        int slot = 0, g = 0, n_tiles = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int gd = 0; ok; ++gd) {
            StepInfo st;
            if (!(ok = take_step(gd, st))) break;
            if (st.N < 0) break;
            if (st.N == 0) continue;
            const bool fresh = st.fresh != 0, last = st.last != 0;
            const uint32_t idesc = st.N == 256 ? idesc_bf16(256, 256, false) : idesc_bf16(256, 128, false);
            const uint32_t d = tmem + (uint32_t)(g & 1) * 256;
            for (int k = 0; k < kSlabs && ok; ++k) {
                // lane 0: Q, lane 1: the keys of a fresh tile, lane 2: D read (step g - 2)
                uint32_t wb = bar(B_QFULL + slot), wp = ph;
                if (lane == 1 && fresh) {
                    wb = bar(B_KFULL + k);
                    wp = (uint32_t)(n_tiles & 1);
                }
                if (lane == 2 && k == 0 && g >= 2) {
                    wb = bar(B_DFREE + (g & 1));
                    wp = (uint32_t)(((g - 2) >> 1) & 1);
                }
                ok = wait_lanes(wb, wp, abort_flag, 2100 + k, g, kApartNs);
                if (!ok) break;
                tc_fence_after();
                const uint64_t ak = d_k + (uint64_t)(k * (kKSlab >> 4)), bq = d_q + (uint64_t)(slot * (kQSlot >> 4));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_pair_ss(d, ak + kk * 2, bq + kk * 2, idesc, (k > 0 || kk > 0) ? 1u : 0u, el);
                issued_any = true;
                mma_commit_pair(bar(B_QEMPTY + slot), el);
                if (last) mma_commit_pair(bar(B_KEMPTY + k), el);
                if (++slot == kQSlots) {
                    slot = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) break;
            mma_commit_pair(bar(B_DFULL + (g & 1)), el);
            if (last) ++n_tiles;
            ++g;
        }
    } else if (warp == 10) {
        // ----------------------------------------------------------- steps
        float* col_f = reinterpret_cast<float*>(sgen + kOffCol);
        StepInfo* info = reinterpret_cast<StepInfo*>(sgen + kOffStep);
        const int sink_end = args.window > 0 ? args.sinks : 0;
        int gd = 0, b_prev = -1, tile_prev = -1, row0 = 0, row1 = 0;
        bool ok = true;
        StepWalk walk(args, ws, cid);
        // the place of step gd
        auto room = [&]() -> bool {
            return ok = wait_lanes(bar(B_STEPFREE + gd % kAhead), (uint32_t)(((gd / kAhead) & 1) ^ 1), abort_flag,
                                   2300, gd, kApartNs);
        };
        // the next step of the walk; steps without work meanwhile, where it takes long
        auto look = [&](Step& s) -> bool {
            while (true) {
                const int found = walk.next(args, ws, s);
                if (found != kStillLooking) return found == kFound;
                if (el) {
                    StepInfo none = {};
                    none.part = -1;
                    info[gd % kAhead] = none;
                    mbar_arrive(bar(B_STEP + gd % kAhead));
                }
                __syncwarp();
                ++gd;
                if (!room()) return false;
            }
        };
        Step cur, nxt;
        room();
        bool have = look(cur);
        while (ok) {
            if (!have) {
                if (el) {
                    info[gd % kAhead].N = -1;
                    mbar_arrive(bar(B_STEP + gd % kAhead));
                }
                break;
            }
            const int N = cur.n > 0 ? n_of(cur) : 0, cols = cur.n * args.Hq;
            // a column's lse and the keys that its row sees (none: a column without a
            // row of this sequence, or with nothing to give)
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = e * 32 + lane;
                v[e] = c < cols ? __ldg(lse + (size_t)cur.t0 * args.Hq + c) : -INFINITY;
            }
            const bool fresh = cur.n > 0 && (cur.b != b_prev || cur.tile != tile_prev);
            if (fresh) {
                b_prev = cur.b;
                tile_prev = cur.tile;
                // blocks of 64 keys behind the last key seen read that key's
                const int* bt = args.pg.block_table + (size_t)cur.b * args.pg.max_pages;
                const int s0 = cur.key0 + 128 * (int)rank, top = cur.hi_b / 64 * 64;
                row0 = (int)key_row(args.pg, bt, 0, min(s0, top));
                row1 = (int)key_row(args.pg, bt, 0, min(s0 + 64, top));
            }
            // a row's keys in its lane; more rows than lanes (fewer than 8 heads): in their columns' lanes
            Visible mine;
            bool live = false;
            if (lane < cur.n) live = sees(args, cur.b, cur.t0 + lane, mine);
            const bool more = look(nxt);
            if (!ok) break;
            const int buf = gd % kAhead;
            float* cl = col_f + buf * 3 * kPairs;
            int* ch = reinterpret_cast<int*>(cl + kPairs);
            int* co = ch + kPairs;
            bool used = true;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = e * 32 + lane, r = min(c / args.Hq, max(cur.n, 1) - 1);
                Visible w;
                bool l;
                if (cur.n <= 32) {
                    w.hi = __shfl_sync(0xffffffffu, mine.hi, r);
                    w.lo = __shfl_sync(0xffffffffu, mine.lo, r);
                    l = __shfl_sync(0xffffffffu, live ? 1 : 0, r) != 0;
                } else {
                    l = sees(args, cur.b, cur.t0 + r, w);
                }
                if (c >= N) continue;
                const bool dead = c >= cols || !l || v[e] == -INFINITY;
                used = used && !dead;
                cl[c] = dead ? 0.f : v[e] * 1.4426950408889634f;
                ch[c] = dead ? -1 : w.hi;
                co[c] = w.lo;
            }
            used = __all_sync(0xffffffffu, used);
            if (el) {
                const int k0 = cur.key0 + 128 * (int)rank;
                StepInfo s;
                s.N = N;
                s.whole = used && cur.n > 0 && k0 + 127 <= cur.rg.min_hi &&
                          (k0 >= cur.rg.max_lo || k0 + 128 <= sink_end);
                s.seen = cur.n > 0 && k0 <= cur.rg.hi && (k0 + 128 > cur.rg.lo || k0 < sink_end);
                s.last = !more || nxt.b != cur.b || nxt.tile != cur.tile;
                s.fresh = fresh;
                s.b = cur.b;
                s.key0 = cur.key0;
                s.part = cur.split ? cid * 2 + (cur.base < walk.w0 ? 0 : 1) : -1;
                s.qrow = cur.t0 * args.Hq;
                s.row[0] = row0;
                s.row[1] = row1;
                info[buf] = s;
                if (rank == 0 && cur.split && s.last) {
                    // the cluster of the tile's last step names it for the join
                    const long long end = cur.base + kTileCost + steps_of(ws.seqs[cur.b], args.Hq);
                    if (end <= walk.w1) {
                        SplitTile d;
                        d.b = cur.b;
                        d.tile = cur.key0;
                        d.c_first = (int)(((cur.base + kTileCost + 1) * walk.ncl - 1) / walk.total);
                        d.c_last = cid;
                        d.base = cur.base;
                        d.total = walk.total;
                        d.ncl = walk.ncl;
                        d.pad = 0;
                        ws.desc[cid] = d;
                    }
                }
            }
            __syncwarp();
            if (el) mbar_arrive(bar(B_STEP + buf));
            cur = nxt;
            have = more;
            ++gd;
            room();
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------- sums
        // TMEM lane i holds key i of this CTA's 128; hs takes half of the columns.
        const int hs = warp >> 2;
        const int i = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const float* col_f = reinterpret_cast<const float*>(sgen + kOffCol);
        const StepInfo* info = reinterpret_cast<const StepInfo*>(sgen + kOffStep);
        float* half_s = reinterpret_cast<float*>(sgen + kOffHalf);
        const uint32_t dfree0 = mapa(bar(B_DFREE), 0);
        const int S = args.pg.max_pages * args.pg.page_size;
        const int sink_end = args.window > 0 ? args.sinks : 0;
        const bool windowed = args.window > 0;
        int g = 0, tiles = 0;
        float sum = 0.f;
        for (int gd = 0;; ++gd) {
            const int at = gd % kAhead;
            if (!wait_all(bar(B_STEP + at), (gd / kAhead) & 1, abort_flag, 2200, gd, kApartNs)) break;
            const StepInfo st = info[at];
            if (st.N < 0) break;
            const int key = st.key0 + 128 * (int)rank + i;
            if (st.N > 0) {
                const float* cl = col_f + at * 3 * kPairs;
                const int* ch = reinterpret_cast<const int*>(cl + kPairs);
                const int* co = ch + kPairs;
                const int buf = g & 1;
                if (!wait_all(bar(B_DFULL + buf), (g >> 1) & 1, abort_flag, 2210, g, kApartNs)) break;
                tc_fence_after();
                const int per = st.N / 2;
                const uint32_t ta = tmem + lane_addr + (uint32_t)buf * 256 + hs * per;
                float acc0 = 0.f, acc1 = 0.f;
#pragma unroll 1
                for (int c0 = 0; c0 < per && st.seen; c0 += 32) {
                    uint32_t d[32];
                    tmem_ld32(ta + c0, d);
                    tmem_wait_ld();
                    const float4* l4 = reinterpret_cast<const float4*>(cl + hs * per + c0);
                    if (st.whole) {
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const float4 l = l4[v];
                            acc0 += ex2(fmaf(__uint_as_float(d[4 * v]), scale_log2, -l.x));
                            acc1 += ex2(fmaf(__uint_as_float(d[4 * v + 1]), scale_log2, -l.y));
                            acc0 += ex2(fmaf(__uint_as_float(d[4 * v + 2]), scale_log2, -l.z));
                            acc1 += ex2(fmaf(__uint_as_float(d[4 * v + 3]), scale_log2, -l.w));
                        }
                    } else {
                        // only the keys that a column's row sees; without a window all of them
                        // from 0 on
                        const int4* h4 = reinterpret_cast<const int4*>(ch + hs * per + c0);
                        const int4* o4 = reinterpret_cast<const int4*>(co + hs * per + c0);
                        auto add = [&](float& acc, uint32_t x, float l, bool seen) {
                            const float p = ex2(fmaf(__uint_as_float(x), scale_log2, -l));
                            if (seen) acc += p;
                        };
                        if (key < sink_end || !windowed) {
#pragma unroll
                            for (int v = 0; v < 8; ++v) {
                                const float4 l = l4[v];
                                const int4 h = h4[v];
                                add(acc0, d[4 * v], l.x, key <= h.x);
                                add(acc1, d[4 * v + 1], l.y, key <= h.y);
                                add(acc0, d[4 * v + 2], l.z, key <= h.z);
                                add(acc1, d[4 * v + 3], l.w, key <= h.w);
                            }
                        } else {
#pragma unroll
                            for (int v = 0; v < 8; ++v) {
                                const float4 l = l4[v];
                                const int4 h = h4[v], o = o4[v];
                                add(acc0, d[4 * v], l.x, key <= h.x && key >= o.x);
                                add(acc1, d[4 * v + 1], l.y, key <= h.y && key >= o.y);
                                add(acc0, d[4 * v + 2], l.z, key <= h.z && key >= o.z);
                                add(acc1, d[4 * v + 3], l.w, key <= h.w && key >= o.w);
                            }
                        }
                    }
                }
                sum += acc0 + acc1;
                tc_fence_before();
                __syncwarp();
                // the loads' results are here, so the signal need not order them
                if (lane == 0) mbar_arrive_remote_relaxed(dfree0 + 8u * (uint32_t)buf);
                ++g;
            }
            if (st.last) {
                // both column halves of a key, then its sum
                float* hv = half_s + tiles % kAhead * 128;
                if (hs == 1) {
                    hv[i] = sum;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_HALF + tiles % kAhead));
                } else {
                    if (!wait_all(bar(B_HALF + tiles % kAhead), (tiles / kAhead) & 1, abort_flag, 2220, g)) break;
                    const float total = sum + hv[i];
                    if (st.part >= 0)
                        ws.parts[(size_t)st.part * kTile + 128 * rank + i] = total;
                    else if (key < S && total != 0.f)
                        mass[(size_t)st.b * S + key] += total;
                }
                sum = 0.f;
                ++tiles;
            }
            // last of all: a tile's buffer of half sums is free by it, too
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_STEPFREE + at));
        }
    }

    if (warp == 9 && issued_any) {
        // every MMA issued completes before TMEM is released
        mma_commit_pair(bar(B_DRAIN), el);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(bar(B_DRAIN), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' MMAs, remote arrivals and copies are over
    tc_fence_after();
    if (warp == 9) tmem_dealloc_pair(tmem, 512);
    cluster_sync();
}

// Adds the partial sums of split tiles, in the order of the clusters.
__global__ void __launch_bounds__(kTile)
cache_mass_join_kernel(const void* ws_raw, int S, float* __restrict__ mass)
{
    griddep_launch();
    griddep_wait();
    const Ws w = ws_of(const_cast<void*>(ws_raw));
    const SplitTile d = w.desc[blockIdx.x];
    if (d.b < 0) return;
    float sum = 0.f;
    for (int c = d.c_first; c <= d.c_last; ++c)
        sum += w.parts[((size_t)c * 2 + (d.base < piece_begin(d.total, d.ncl, c) ? 0 : 1)) * kTile + threadIdx.x];
    const int key = d.tile + (int)threadIdx.x;
    if (key < S && sum != 0.f) mass[(size_t)d.b * S + key] += sum;
}

}  // namespace cache_mass
}  // namespace dsa
