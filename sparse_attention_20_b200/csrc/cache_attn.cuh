// Dense MLA attention (MQA mode) of new tokens over the paged latent cache,
// and the attention weight each cached token receives from it. Row t of
// sequence b = seq[t] at position p = pos[t] sees the keys
//   V(t) = { s <= p },  or with a window W > 0  { s <= p : s > p - W or s < sinks }
// and
//   x_s = scale q[t,h].c_s,  lse = log sum_V exp x_s,
//   out[t,h] = sum_V exp(x_s - lse) c_s[0:512],
//   mass[b,s] += sum over the rows t of b that see s, and h, of exp(x_s - lse[t,h]).
#pragma once
#include "common.cuh"

namespace dsa {
namespace cache_attn {

constexpr int kDqk = 576;
constexpr int kDv = 512;

// Visible keys of a row: [lo, hi] and [0, sink_end) (hi = -1: none).
struct Visible {
    int lo, hi, sink_end;
    __device__ __forceinline__ bool operator()(int s) const { return s <= hi && (s >= lo || s < sink_end); }
};

__device__ __forceinline__ Visible visible_of(int n_keys, int pos, int window, int sinks)
{
    Visible v;
    v.hi = n_keys - 1;
    v.lo = window > 0 && pos >= window ? pos - window + 1 : 0;
    v.sink_end = window > 0 ? sinks : 0;
    return v;
}

// One warp per (sequence, key), over the sequence's rows and heads.
__global__ void __launch_bounds__(256)
mla_attn_mass_simple_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ kv,
                            const PagedRows pg, const int* __restrict__ pos, const float* __restrict__ lse, int T,
                            int Hq, float scale, int window, int sinks, float* __restrict__ mass)
{
    const int lane = threadIdx.x & 31;
    const int S = pg.max_pages * pg.page_size;
    const long long key = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (key >= (long long)pg.n_seqs * S) return;
    const int b = (int)(key / S), s = (int)(key % S);
    float2 cv[9];
    bool have = false;
    float sum = 0.f;
    for (int t = 0; t < T; ++t) {
        if (pg.seq[t] != b) continue;
        long long base;
        const int* bt;
        const int n = row_keys(pg, pos, nullptr, t, T, 0, &base, &bt);
        if (!visible_of(n, pos[t], window, sinks)(s)) continue;
        if (!have) {
            const __nv_bfloat162* c = reinterpret_cast<const __nv_bfloat162*>(kv + key_row(pg, bt, base, s) * kDqk);
            for (int i = 0; i < 9; ++i) cv[i] = __bfloat1622float2(c[i * 32 + lane]);
            have = true;
        }
        for (int h = 0; h < Hq; ++h) {
            const size_t row = (size_t)t * Hq + h;
            float x = 0.f;
            for (int i = 0; i < 9; ++i) {
                const float2 qv = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(q + row * kDqk)[i * 32 + lane]);
                x = fmaf(qv.x, cv[i].x, fmaf(qv.y, cv[i].y, x));
            }
            for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            const float ls = lse[row];
            if (ls != -INFINITY) sum += expf(x * scale - ls);
        }
    }
    if (have && lane == 0) mass[key] += sum;
}

}  // namespace cache_attn
}  // namespace dsa
