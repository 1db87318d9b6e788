// kda_qk_norm.cu -- the norm of queries and keys per head with the position rotation in the same
// pass, forward and backward.
//
//   n = x c,  c = (mean x^2 + eps)^-1/2,  y = rot(w n)          per (token, head) of d channels
//   rot turns pair i of the first 2 R channels, (i, R + i) or interleaved (2 i, 2 i + 1), by the
//   angle position * freqs[i]
//   backward: u = rot^-1(dy), t = w u:  dx = c (t - n mean(t n)),  dw = sum over tokens and heads of u n
//
// Angles: a frequency is held as the fraction of a turn per position in 64-bit fixed point; times the
// position, modulo 2^64, it is the angle's fraction of a turn to 2^-64 of a turn per position, whatever
// the position's size or sign, by integer products alone (fp64 is narrow on this part).
// Both passes are bound by HBM: every input is read once and kept in registers across its row's
// sums. A CTA takes a few tokens at a time: its threads form the tokens' sines and cosines in shared
// memory, a pair each, which all heads then share; groups of threads walk over the rows (token,
// head). Sums over rows go to one partial row a CTA and are added up by a second kernel in a fixed
// order: the same call gives the same bits.
#include <cuda_bf16.h>

#include <algorithm>

#include "kda_internal.h"
#include "kda_ptx.h"

namespace kda {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 256;
constexpr int kMaxD = 256;

__device__ __forceinline__ float get(const float *p) { return *p; }
__device__ __forceinline__ float get(const bf16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(bf16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void load8(const float *p, float *x) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16 *p, float *x) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float *x) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(bf16 *p, const float *x) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(ptx::pack_bf16(x[0], x[1]), ptx::pack_bf16(x[2], x[3]),
                                               ptx::pack_bf16(x[4], x[5]), ptx::pack_bf16(x[6], x[7]));
}

// The fraction of a turn that a position adds to a pair's angle
__device__ __forceinline__ uint64_t turn_fraction(double freq) {
    const double t = freq * 0.15915494309189535;  // 1 / (2 pi)
    const double f = t - floor(t);                // in [0, 1]: 1 only by rounding, and then 0
    return f >= 1.0 ? 0 : (uint64_t)(f * 18446744073709551616.0);
}
__device__ __forceinline__ float2 cos_sin(uint64_t turn) {
    float2 cs;
    // half turns in [-1, 1), to 2^-31 of one before its rounding to fp32
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &cs.y, &cs.x);
    return cs;
}

// A group of G threads (a power of two up to 32) holds a row of d channels, eight a thread: with
// VEC thread t the run 8 t .., otherwise the channels t + G i.
template <bool VEC>
__device__ __forceinline__ int channel(int t, int G, int i) { return VEC ? 8 * t + i : t + G * i; }

template <bool VEC, typename T>
__device__ __forceinline__ void load_row(const T *p, int d, int t, int G, float *x) {
    if constexpr (VEC) {
        if (8 * t < d) {
            load8(p + 8 * t, x);
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = t + G * i < d ? get(p + t + G * i) : 0.f;
    }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_row(T *p, int d, int t, int G, const float *x) {
    if constexpr (VEC) {
        if (8 * t < d) store8(p + 8 * t, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t + G * i < d) put(p + t + G * i, x[i]);
    }
}
__device__ __forceinline__ float group_sum(float x, int G) {
    for (int o = G >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The row x turned by the token's angles (sign = -1: back). cs: the token's (cos, sin) pairs;
// stage: d floats of this group. Every thread of the warp calls it.
template <bool VEC>
__device__ __forceinline__ void turn(float *x, const float2 *cs, int R, bool interleaved, float sign, int t, int G,
                                     float *stage) {
    if (VEC && interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const int c = 8 * t + i;
            if (c < 2 * R) {
                const float2 a = cs[c >> 1];
                const float s = sign * a.y, y = x[i] * a.x - x[i + 1] * s;
                x[i + 1] = fmaf(x[i + 1], a.x, x[i] * s);
                x[i] = y;
            }
        }
        return;
    }
    if (VEC && (R & 7) == 0) {  // a run's partners are another thread's run
        const int by = R >> 3, lane = threadIdx.x & 31;
        const bool low = t < by, in = t < 2 * by;
        const int from = in ? (low ? lane + by : lane - by) : lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float other = __shfl_sync(0xffffffffu, x[i], from);
            if (in) {
                const float2 a = cs[8 * (low ? t : t - by) + i];
                x[i] = fmaf(low ? -other : other, sign * a.y, x[i] * a.x);
            }
        }
        return;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (channel<VEC>(t, G, i) < 2 * R) stage[channel<VEC>(t, G, i)] = x[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = channel<VEC>(t, G, i);
        if (c < 2 * R) {
            const bool low = interleaved ? (c & 1) == 0 : c < R;
            const int pair = interleaved ? c >> 1 : low ? c : c - R;
            const float other = stage[interleaved ? c ^ 1 : low ? c + R : c - R];
            const float2 a = cs[pair];
            x[i] = fmaf(low ? -other : other, sign * a.y, x[i] * a.x);
        }
    }
}

__device__ __forceinline__ int64_t position(const QkNormArgs &p, int64_t t) {
    return p.wide_positions ? static_cast<const int64_t *>(p.positions)[t] : static_cast<const int32_t *>(p.positions)[t];
}

// A CTA takes `tokens` tokens at a time, every gridDim.x-th of such blocks. Dynamic shared memory:
// the pairs' fractions of a turn, the tokens' (cos, sin) [tokens][R], the groups' stages.
struct Layout {
    int tokens, G;
    __host__ __device__ size_t angles(int R) const { return 8 * (size_t)R; }
    __host__ __device__ size_t stages(int R) const { return angles(R) + (size_t)tokens * R * 8; }
    __host__ __device__ size_t bytes(int R, bool staged) const {
        return stages(R) + (staged ? (size_t)kThreads / G * 2 * R * 4 : 0);
    }
};

template <typename T, bool VEC, bool BWD>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const QkNormArgs p, const Layout l) {
    extern __shared__ __align__(16) char smem[];
    uint64_t *frac = reinterpret_cast<uint64_t *>(smem);
    float2 *cs = reinterpret_cast<float2 *>(smem + l.angles(p.n_freqs));
    const int R = p.n_freqs, G = l.G, groups = kThreads / G;
    const int tid = threadIdx.x, group = tid / G, t = tid % G;
    float *stage = reinterpret_cast<float *>(smem + l.stages(R)) + group * 2 * R;
    const int heads = p.heads[0] + p.heads[1];
    for (int i = tid; i < R; i += kThreads) frac[i] = turn_fraction(p.freqs[i]);
    float w[2][8];
#pragma unroll
    for (int n = 0; n < 2; ++n) load_row<VEC>(p.weight[n], p.d, t, G, w[n]);
    float dw[2][8];
    if constexpr (BWD)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[n][i] = 0.f;
    const float inv_d = 1.f / p.d;
    for (int64_t t0 = (int64_t)blockIdx.x * l.tokens; t0 < p.n_tok; t0 += (int64_t)gridDim.x * l.tokens) {
        const int n_tok = (int)min((int64_t)l.tokens, p.n_tok - t0);
        __syncthreads();
        for (int i = tid; i < n_tok * R; i += kThreads) {
            const int tok = i / R;
            cs[i] = cos_sin(frac[i - tok * R] * (uint64_t)position(p, t0 + tok));
        }
        __syncthreads();
        const int rows = n_tok * heads, rounds = (rows + groups - 1) / groups;
        for (int n = 0; n < rounds; ++n) {
            const int row = n * groups + group;
            const bool live = row < rows;
            const int tok = live ? row / heads : 0, h = live ? row - tok * heads : 0;
            const int which = h >= p.heads[0], head = which ? h - p.heads[0] : h;
            float x[8], u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = u[i] = 0.f;
            if (live) {
                load_row<VEC>(static_cast<const T *>(p.x[which]) + (t0 + tok) * p.stride[which] + (int64_t)head * p.d, p.d, t, G, x);
                if constexpr (BWD)
                    load_row<VEC>(static_cast<const T *>(p.dy[which]) + (t0 + tok) * p.dy_stride[which] + (int64_t)head * p.d, p.d, t, G, u);
            }
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
            ss = group_sum(ss, G);
            const float c = 1.f / sqrtf(ss * inv_d + p.eps);
            T *y = static_cast<T *>(p.y[which]) + ((t0 + tok) * p.heads[which] + head) * p.d;
            if constexpr (!BWD) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= c * (which ? w[1][i] : w[0][i]);
                turn<VEC>(x, cs + tok * R, R, p.interleaved, 1.f, t, G, stage);
                if (live) store_row<VEC>(y, p.d, t, G, x);
            } else {
                turn<VEC>(u, cs + tok * R, R, p.interleaved, -1.f, t, G, stage);
                float tn = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] *= c;
                    const float un = u[i] * x[i];
                    if (which) dw[1][i] += un;
                    else dw[0][i] += un;
                    u[i] *= which ? w[1][i] : w[0][i];
                    tn = fmaf(u[i], x[i], tn);
                }
                tn = group_sum(tn, G) * inv_d;
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = c * (u[i] - x[i] * tn);
                if (live) store_row<VEC>(y, p.d, t, G, u);
            }
        }
    }
    if constexpr (BWD) {  // the groups' sums, in a fixed order
        __shared__ float sum[kThreads / 32][kMaxD];
        // groups of a warp first, then the warps
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float x = dw[n][i];
                for (int o = G; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                const int c = channel<VEC>(t, G, i);
                if ((tid & 31) < G && c < p.d) sum[tid >> 5][c] = x;
            }
            __syncthreads();
            for (int c = tid; c < p.d; c += kThreads) {
                float x = 0.f;
#pragma unroll
                for (int i = 0; i < kThreads / 32; ++i) x += sum[i][c];
                p.partial[((int64_t)n * gridDim.x + blockIdx.x) * p.d + c] = x;
            }
        }
    }
}

// dw[n][c] = the sum of the partial rows: a warp per channel column, rows dealt out to its lanes
__global__ void __launch_bounds__(kThreads) qk_norm_sum_kernel(const float *partial, int rows, int d, float *dq, float *dk) {
    const int n = blockIdx.y, c0 = blockIdx.x * 32, c = c0 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    __shared__ float sum[kThreads / 32][32];
    float x = 0.f;
    if (c < d)
        for (int i = part; i < rows; i += kThreads / 32) x += partial[((int64_t)n * rows + i) * d + c];
    sum[part][threadIdx.x & 31] = x;
    __syncthreads();
    if (part == 0 && c < d) {
        x = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) x += sum[i][threadIdx.x];
        (n ? dk : dq)[c] = x;
    }
}

constexpr int kBwdBlocks = 152 * 4;

template <typename T>
bool vector_rows(const QkNormArgs &p, bool bwd) {
    if (p.d % 8 != 0) return false;
    for (int i = 0; i < 2; ++i) {
        const void *ptrs[] = {p.x[i], p.y[i], bwd ? p.dy[i] : nullptr};
        for (const void *x : ptrs)
            if ((uintptr_t)x % 16 != 0) return false;
        if ((uintptr_t)p.weight[i] % 16 != 0) return false;
        if (p.stride[i] * sizeof(T) % 16 != 0 || (bwd && p.dy_stride[i] * sizeof(T) % 16 != 0)) return false;
    }
    return true;
}

template <typename T, bool BWD>
cudaError_t run(const QkNormArgs &p, cudaStream_t stream) {
    const int heads = p.heads[0] + p.heads[1];
    Layout l;
    l.G = 1;
    while (8 * l.G < p.d) l.G *= 2;
    // as many tokens as give every group a few rows, and every thread a sine
    const int groups = kThreads / l.G;
    l.tokens = std::max(1, std::min(16, 8 * groups / heads));
    const int64_t blocks = (p.n_tok + l.tokens - 1) / l.tokens;
    const unsigned grid = (unsigned)(BWD ? std::min<int64_t>(blocks, kBwdBlocks) : std::min<int64_t>(blocks, 0x7fffffff));
    const bool vec = vector_rows<T>(p, BWD);
    const bool staged = !(vec && (p.interleaved || p.n_freqs % 8 == 0));
    const size_t smem = l.bytes(p.n_freqs, staged);
    if (grid > 0) {
        if (vec) qk_norm_kernel<T, true, BWD><<<grid, kThreads, smem, stream>>>(p, l);
        else qk_norm_kernel<T, false, BWD><<<grid, kThreads, smem, stream>>>(p, l);
        count_launches(1);
    }
    if (BWD) {
        qk_norm_sum_kernel<<<dim3((p.d + 31) / 32, 2), kThreads, 0, stream>>>(p.partial, (int)grid, p.d, p.dw[0], p.dw[1]);
        count_launches(1);
    }
    return cudaGetLastError();
}

}  // namespace

size_t qk_norm_workspace_bytes(int64_t n_tok, int32_t d) {
    return (size_t)std::min<int64_t>(n_tok, kBwdBlocks) * 2 * d * 4;
}

cudaError_t launch_qk_norm(const QkNormArgs &p, bool bwd, cudaStream_t stream) {
    if (p.bf16) return bwd ? run<bf16, true>(p, stream) : run<bf16, false>(p, stream);
    return bwd ? run<float, true>(p, stream) : run<float, false>(p, stream);
}

}  // namespace kda
