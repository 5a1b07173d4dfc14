// What dense MLA attention (MQA mode) of new tokens over the paged latent cache
// and the weight each cached token receives from it have in common. Row t of
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
};

__device__ __forceinline__ Visible visible_of(int n_keys, int pos, int window, int sinks)
{
    Visible v;
    v.hi = n_keys - 1;
    v.lo = window > 0 && pos >= window ? pos - window + 1 : 0;
    v.sink_end = window > 0 ? sinks : 0;
    return v;
}

}  // namespace cache_attn
}  // namespace dsa
