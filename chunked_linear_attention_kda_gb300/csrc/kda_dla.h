// Shared by the kernels of linear attention with one decay per head (kda_dla_*.cu): chunk slots
// and a chunk's decays. Internal; not part of the C ABI.
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = s S_t^T q_t
//
// Over a chunk of C tokens with start state S0, D_rj = sum of g over (j, r], e = e^D for r >= j
// (else 0), gamma_r the decay up to and with r, delta_j the decay past j, Gamma of all:
//   O = s (gamma Q S0 + (e Q K^T) V),   S1 = Gamma S0 + (delta K)^T V
// and backward, with the gradient dS1 of the end state and W = s e (dO V^T):
//   dS0 = Gamma dS1 + s (gamma Q)^T dO
//   dQ = s gamma dO S0^T + W K,   dK = delta V dS1^T + W^T Q
//   dV = delta K dS1 + (s e Q K^T)^T dO
//   dg_t = Gamma <S0, dS1> + sum_{r >= t} a_r + sum_{j < t} b_j + sum_{j < t <= r} W_rj q_r.k_j
//   a_r = s gamma_r q_r.(S0 dO_r),  b_j = delta_j k_j.(dS1 v_j);  the double sum is a running sum of
//   row sums minus column sums.
// No exponent above zero is formed: decays may be as strong as they like. g below -200 (and -inf, a
// reset) is a decay of 0 in fp32 and acts as -inf; dg there is 0.
#pragma once

#include "kda_gdr.h"

namespace kda {
namespace dla {

using gdr::add;
using gdr::Chunk;
using gdr::ex2;
using gdr::find_chunk;
using gdr::kGFloor;
using gdr::n_slots;
using gdr::slot_base;
using gdr::Two;

// log2(e) in two floats
constexpr float kLog2e = 1.44269502f, kLog2eLo = 1.92596299e-8f;

// g log2(e) as two floats
__device__ __forceinline__ Two decay_exponent(float g) {
    const float x = g < kGFloor ? kGFloor : g;  // finite: no inf - inf in differences of sums
    const float hi = x * kLog2e;
    return {hi, fmaf(x, kLog2e, -hi) + x * kLog2eLo};
}
__device__ __forceinline__ Two minus(Two x, Two y) { return add(x, {-y.hi, -y.lo}); }
__device__ __forceinline__ Two up(Two x, int o) {
    return {__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
}
// inclusive sums over a warp's lanes
__device__ __forceinline__ Two warp_scan(Two x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two y = up(x, o);
        if (lane >= o) x = add(y, x);
    }
    return x;
}
__device__ __forceinline__ Two last_lane(Two x) {
    return {__shfl_sync(0xffffffffu, x.hi, 31), __shfl_sync(0xffffffffu, x.lo, 31)};
}
// 2^(hi + lo), lo small beside 1
__device__ __forceinline__ float exp2_of(Two x) {
    const float e = ex2(x.hi);
    return fmaf(e * 0.693147181f, x.lo, e);
}
// 2^(n + f), n whole, f up to 1/2 of either sign, in two floats: near 1 what the decay takes away has 23 bits
// of its own.
__device__ __forceinline__ Two exp2_parts(float n, float f) {
    const float e = ex2(n), m = expm1f(f * 0.693147181f), w = 1.f + m;
    return {e * w, e * (m - (w - 1.f))};
}
// The decays that multiply a state one after the other. Near 1 a float is off by up to 2^-25, and with a
// constant rate by the same amount every time, which adds up over the memory (64K tokens in tiles of 64 at
// rates of 1e-6: the state off by 4e-5 of its norm). So what a factor's rounding left out, relative to it, goes
// to the next factor: a product over any run is off by one rounding at its start and one at its end. Below
// 1/4 nothing is handed on: what is left of a state does not add up.
struct Factors {
    float owed = 0.f;
    __device__ __forceinline__ float next(Two decay) {
        const float more = fmaf(decay.hi, owed, decay.lo), w = decay.hi + more;
        owed = w > 0.25f ? __fdividef((decay.hi - w) + more, w) : 0.f;
        return w;
    }
};
// 2^(a - b) for neighbouring sums
__device__ __forceinline__ float exp2_between(float2 a, float2 b) { return ex2((a.x - b.x) + (a.y - b.y)); }

// dg[head] = the sum of a column of sums [rows, heads], in a fixed order
cudaError_t launch_dla_sum_decay(const float *sums, int64_t rows, int heads, float *dg, cudaStream_t stream);

}  // namespace dla

// fp32 inputs, and calls without a token: kernels without tensor cores (kda_dla_simt.cu).
size_t dla_simt_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k, int32_t d_v, bool bwd);
cudaError_t launch_dla_simt(const DlaArgs &args, bool bwd, cudaStream_t stream);
// bf16 inputs: tcgen05 (kda_dla_fwd.cu, kda_dla_bwd.cu).
size_t dla_tc_fwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k, int32_t d_v);
cudaError_t launch_dla_tc_fwd(const DlaArgs &args, cudaStream_t stream);
size_t dla_tc_bwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k, int32_t d_v);
cudaError_t launch_dla_tc_bwd(const DlaArgs &args, cudaStream_t stream);

}  // namespace kda
