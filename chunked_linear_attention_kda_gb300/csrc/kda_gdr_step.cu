// kda_gdr_step.cu -- one token of the gated delta rule with one decay per head, for a batch
// of sequences whose states live in a pool: row b updates state[slots[b]] in place.
//
//   S' = exp(g) S;  u = beta (v - S'^T k);  S <- S' + k u^T;  o = d_k^-1/2 S^T q
//      = d_k^-1/2 (S'^T q + (q . k) u)
//
// Column j of S needs only its own dot products with k and q before it is rewritten: the
// state is read once and written once, 8 d_k d_v bytes against 7 d_k d_v flops, so HBM
// bounds it: 253 rows of 32 heads, 1.03 GB, take 159 us, 0.96 of a plain copy's bandwidth. A thread keeps its part of the state (R rows of VEC columns) in registers
// between the read and the write.
#include <cuda_bf16.h>

#include <cmath>

#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxK = 128;

__device__ __forceinline__ float get(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float get(const __nv_bfloat16 *p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void put(float *p, int64_t i, float x) { p[i] = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, int64_t i, float x) { p[i] = __float2bfloat16_rn(x); }

// CB columns of one (row, head) per CTA.
template <typename T, int CB, int VEC>
__global__ void __launch_bounds__(kThreads)
    gdr_step_kernel(const GdrStepArgs p, float scale) {
    constexpr int TC = CB / VEC;            // threads across the columns
    constexpr int RB = kThreads / TC;       // row blocks
    constexpr int R = kMaxK / RB;           // rows of a thread
    __shared__ float ks[kMaxK], qs[kMaxK], part[RB][2][CB], ucol[CB], qk_warp[kMaxK / 32];
    const int n_blk = (p.d_v + CB - 1) / CB;
    const int blk = blockIdx.x % n_blk;
    const int64_t bh = blockIdx.x / n_blk;
    const int head = (int)(bh % p.n_heads), kh = head / (p.n_heads / p.n_k_heads);
    const int64_t b = bh / p.n_heads;
    const int t = threadIdx.x, j0 = blk * CB;
    const int64_t slot = p.slots ? p.slots[b] : b;
    T *out = static_cast<T *>(p.out) + bh * p.d_v + j0;
    if (slot < 0 || slot >= p.n_slots) {  // a padded row
        if (t < CB && j0 + t < p.d_v) put(out, t, 0.f);
        return;
    }
    const int c = (t % TC) * VEC, r0 = (t / TC) * R;
    const int rows = j0 + c < p.d_v ? min(R, p.d_k - r0) : 0;
    float *S = p.state + ((slot * p.n_heads + head) * p.d_k + r0) * p.d_v + j0 + c;
    float s[R][VEC];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (i < rows) {
            if constexpr (VEC == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(S + (int64_t)i * p.d_v);
                s[i][0] = x.x; s[i][1] = x.y; s[i][2] = x.z; s[i][3] = x.w;
            } else {
                s[i][0] = S[(int64_t)i * p.d_v];
            }
        } else {
#pragma unroll
            for (int x = 0; x < VEC; ++x) s[i][x] = 0.f;
        }
    }
    const float decay = expf(p.g[bh]);
    if (t < kMaxK) {
        float kc = 0.f, qc = 0.f;
        if (t < p.d_k) {
            kc = get(static_cast<const T *>(p.k), b * p.k_stride + (int64_t)kh * p.d_k + t);
            qc = get(static_cast<const T *>(p.q), b * p.q_stride + (int64_t)kh * p.d_k + t);
        }
        ks[t] = kc;
        qs[t] = qc;
        float x = kc * qc;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if ((t & 31) == 0) qk_warp[t >> 5] = x;
    }
    __syncthreads();
    float pk[VEC], pq[VEC];
#pragma unroll
    for (int x = 0; x < VEC; ++x) pk[x] = pq[x] = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float kc = ks[r0 + i], qc = qs[r0 + i];
#pragma unroll
        for (int x = 0; x < VEC; ++x) {
            s[i][x] *= decay;
            pk[x] = fmaf(kc, s[i][x], pk[x]);
            pq[x] = fmaf(qc, s[i][x], pq[x]);
        }
    }
#pragma unroll
    for (int x = 0; x < VEC; ++x) {
        part[t / TC][0][c + x] = pk[x];
        part[t / TC][1][c + x] = pq[x];
    }
    __syncthreads();
    if (t < CB && j0 + t < p.d_v) {
        float yk = 0.f, yq = 0.f;
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            yk += part[i][0][t];
            yq += part[i][1][t];
        }
        const float qk = (qk_warp[0] + qk_warp[1]) + (qk_warp[2] + qk_warp[3]);
        const float v = get(static_cast<const T *>(p.v), b * p.v_stride + (int64_t)head * p.d_v + j0 + t);
        const float u = p.beta[bh] * (v - yk);
        ucol[t] = u;
        put(out, t, scale * fmaf(qk, u, yq));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (i >= rows) break;
        const float kc = ks[r0 + i];
        if constexpr (VEC == 4) {
            *reinterpret_cast<float4 *>(S + (int64_t)i * p.d_v) =
                make_float4(fmaf(kc, ucol[c], s[i][0]), fmaf(kc, ucol[c + 1], s[i][1]),
                            fmaf(kc, ucol[c + 2], s[i][2]), fmaf(kc, ucol[c + 3], s[i][3]));
        } else {
            S[(int64_t)i * p.d_v] = fmaf(kc, ucol[c], s[i][0]);
        }
    }
}

template <typename T, int CB, int VEC>
void run(const GdrStepArgs &p, float scale, cudaStream_t stream) {
    const unsigned grid = (unsigned)((p.d_v + CB - 1) / CB) * p.n_rows * p.n_heads;
    gdr_step_kernel<T, CB, VEC><<<grid, kThreads, 0, stream>>>(p, scale);
}

// 128 columns to a CTA read whole rows of the state; with few (row, head) pairs 32 columns keep
// more SMs busy. At d_k = d_v = 128: 32 pairs 3.0 us with 32 columns, 3.9 with 128; 64 pairs 3.5
// and 3.9; 128 pairs 4.8 and 4.2; 256 pairs 6.7 and 6.1; 8096 pairs 184 and 162 us.
template <typename T>
void pick(const GdrStepArgs &p, float scale, cudaStream_t stream) {
    const bool vec = p.d_v % 4 == 0 && ((uintptr_t)p.state & 15u) == 0;
    if (!vec) run<T, 32, 1>(p, scale, stream);
    else if ((int64_t)p.n_rows * p.n_heads < 128) run<T, 32, 4>(p, scale, stream);
    else run<T, 128, 4>(p, scale, stream);
}

}  // namespace

cudaError_t launch_gdr_step(const GdrStepArgs &p, cudaStream_t stream) {
    const float scale = 1.f / std::sqrt((float)p.d_k);
    if (p.bf16) pick<__nv_bfloat16>(p, scale, stream);
    else pick<float>(p, scale, stream);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace kda
