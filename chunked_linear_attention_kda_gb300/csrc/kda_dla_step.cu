// kda_dla_step.cu -- one token of linear attention with one decay per head, for a batch of sequences
// whose states live in a pool: row b updates state[slots[b]] in place.
//
//   S <- e^g S + k v^T,   o = s S^T q
//
// The state is read once and written once, 8 d_k d_v bytes against 5 d_k d_v flops: HBM bounds it. The
// output needs a sum over the state's rows, the update does not: a thread writes its part of the
// state back before the sum over threads. A head's columns are dealt out in runs of VEC, rows of runs
// to consecutive threads, so that a warp's reads are contiguous whatever d_v. 253 rows of 32 heads, 128 x 128:
// 154 us, the copy rate.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxK = 128;

__device__ __forceinline__ float get(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float get(const __nv_bfloat16 *p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void put(float *p, int64_t i, float x) { p[i] = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, int64_t i, float x) { *(p + i) = __float2bfloat16_rn(x); }

// A CTA holds `cols` columns (a multiple of VEC) of one (row, head): thread t has the columns
// VEC (t % TC) .. of the rows t / TC, t / TC + RB, ..; R bounds its rows.
template <typename T, int R, int VEC>
__global__ void __launch_bounds__(kThreads) dla_step_kernel(const DlaStepArgs p, int cols) {
    __shared__ float ks[kMaxK], qs[kMaxK], part[kThreads * VEC];
    const int n_blk = (p.d_v + cols - 1) / cols;
    const int blk = blockIdx.x % n_blk;
    const int64_t bh = blockIdx.x / n_blk;
    const int head = (int)(bh % p.n_heads), kh = head / (p.n_heads / p.n_k_heads);
    const int64_t b = bh / p.n_heads;
    const int t = threadIdx.x, j0 = blk * cols, width = min(cols, p.d_v - j0);
    const int TC = width / VEC, RB = kThreads / TC;
    const int64_t slot = p.slots ? p.slots[b] : b;
    T *out = static_cast<T *>(p.out) + bh * p.d_v + j0;
    if (slot < 0 || slot >= p.n_slots) {  // a padded row
        if (t < width) put(out, t, 0.f);
        return;
    }
    const int c = (t % TC) * VEC, r0 = t / TC;
    const int rows = r0 < RB ? (p.d_k - r0 + RB - 1) / RB : 0;
    const int64_t step = (int64_t)RB * p.d_v;
    float *S = p.state + ((slot * p.n_heads + head) * p.d_k + r0) * p.d_v + j0 + c;
    float s[R][VEC];
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < rows) {
            if constexpr (VEC == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(S + i * step);
                s[i][0] = x.x; s[i][1] = x.y; s[i][2] = x.z; s[i][3] = x.w;
            } else {
                s[i][0] = S[i * step];
            }
        }
    // The decay in two parts: a float beside 1 is off by up to 2^-25, with a constant rate by the same amount at
    // every token, which adds up (4096 tokens at g = -1e-4: the state by 8e-5 of its norm).
    const float g = p.g[b * p.g_stride + head];
    float decay = expf(g), rest = 0.f;
    if (g > -0.5f) {  // a branch: selected from both, 253 rows take 156 us
        const float less = expm1f(g);
        decay = 1.f + less;
        rest = less - (decay - 1.f);
    }
    if (decay == 0.f)  // what is forgotten may be anything: a NaN that the slot's last owner left
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int x = 0; x < VEC; ++x) s[i][x] = 0.f;
    float v[VEC], o[VEC];
#pragma unroll
    for (int x = 0; x < VEC; ++x) {
        v[x] = get(static_cast<const T *>(p.v), b * p.v_stride + (int64_t)head * p.d_v + j0 + c + x);
        o[x] = 0.f;
    }
    if (t < p.d_k) {
        ks[t] = get(static_cast<const T *>(p.k), b * p.k_stride + (int64_t)kh * p.d_k + t);
        qs[t] = get(static_cast<const T *>(p.q), b * p.q_stride + (int64_t)kh * p.d_k + t);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (i >= rows) break;
        const float kc = ks[r0 + i * RB], qc = qs[r0 + i * RB];
#pragma unroll
        for (int x = 0; x < VEC; ++x) {
            const float y = fminf(fmaxf(s[i][x], -FLT_MAX), FLT_MAX);  // no 0 times an infinity: that stays one
            s[i][x] = fmaf(decay, s[i][x], fmaf(kc, v[x], rest * y));
            o[x] = fmaf(qc, s[i][x], o[x]);
        }
        if constexpr (VEC == 4) *reinterpret_cast<float4 *>(S + i * step) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
        else S[i * step] = s[i][0];
    }
    if (r0 < RB) {
#pragma unroll
        for (int x = 0; x < VEC; ++x) part[r0 * width + c + x] = o[x];
    }
    __syncthreads();
    if (t < width) {
        float y = 0.f;
        for (int i = 0; i < RB; ++i) y += part[i * width + t];
        put(out, t, p.scale * y);
    }
}

template <typename T, int R, int VEC>
void run(const DlaStepArgs &p, int cols, cudaStream_t stream) {
    const unsigned grid = (unsigned)((p.d_v + cols - 1) / cols) * p.n_rows * p.n_heads;
    dla_step_kernel<T, R, VEC><<<grid, kThreads, 0, stream>>>(p, cols);
}

// Whole rows of the state to a CTA; with few (row, head) pairs 32 columns keep more SMs busy.
template <typename T>
void pick(const DlaStepArgs &p, cudaStream_t stream) {
    if (p.d_v % 4 == 0 && ((uintptr_t)p.state & 15u) == 0) {
        const int cols = (int64_t)p.n_rows * p.n_heads < 128 ? std::min(32, (int)p.d_v) : p.d_v;
        const int rows = (p.d_k + kThreads / (cols / 4) - 1) / (kThreads / (cols / 4));
        if (rows <= 4) run<T, 4, 4>(p, cols, stream);
        else if (rows <= 8) run<T, 8, 4>(p, cols, stream);
        else run<T, 16, 4>(p, cols, stream);
    } else {
        const int cols = std::min(32, (int)p.d_v);
        run<T, 16, 1>(p, cols, stream);
    }
}

}  // namespace

cudaError_t launch_dla_step(const DlaStepArgs &p, cudaStream_t stream) {
    if (p.bf16) pick<__nv_bfloat16>(p, stream);
    else pick<float>(p, stream);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace kda
