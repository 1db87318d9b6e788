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
// Every input is read once and kept across its row's sums. bf16 rows by loads of four or two are in registers
// (backward all but 40 to 160 bytes a thread), and HBM bounds the forward pass. fp32 rows and rows by single
// channels take twice the registers, and part of them goes to local memory and back (fp32: 64K tokens of 32 + 8
// heads of 128 channels 591 us, 0.68 of the copy rate; backward of 8191 of 32 + 32 heads 185 us, 0.65).
// Groups of threads hold rows; a warp's groups take the heads of one token in turn, so that its angles are
// formed once and stay in registers, and a thread holds both channels of each of its pairs, so that
// none goes through shared memory (a first form, with a run of channels a thread and the angles in shared
// memory, was bound by that: 511 us at 64K tokens of 32 + 8 heads of 128 channels, 224 so, 0.90 of the copy
// rate; backward of 8191 tokens of 32 + 32 heads 95 us, 0.64, with the conversions and sums in 0.57 of the issue slots). Sums over rows go to one partial row a CTA
// and are added up by a second kernel in a fixed order: the same call gives the same bits.
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

// A group of G threads (a power of two up to 32) holds a row of d channels, eight a thread: both channels
// of four pairs, by loads of four channels or, where the row's length, its halves or its address allow no more, of
// two; otherwise (odd lengths or halves) the channels t + G i, and the pairs meet in shared memory. 20000
// tokens of 32 + 32 heads of 100 channels, backward: 1160 us by single channels, 238 by two.
enum Kind { kSingle, kHalves, kInterleaved, kHalves2, kInterleaved2 };
__host__ __device__ constexpr int width(Kind k) { return k == kSingle ? 1 : k == kHalves || k == kInterleaved ? 4 : 2; }
__host__ __device__ constexpr bool interleaves(Kind k) { return k == kInterleaved || k == kInterleaved2; }
// Where the thread's channels 0 and 1, 2 and 3, 4 and 5, 6 and 7 lie. Loads of four: pairs from 4 t on (halves: beyond
// the pairs two runs side by side). Loads of two: the slots t and t + G of two pairs each, or of four
// channels side by side beyond the pairs.
struct Runs { int a, a2, b, b2; };
template <Kind KIND>
__device__ __forceinline__ Runs runs(int t, int R, int G) {
    if constexpr (width(KIND) == 2) {
        auto slot = [&](int s) { return interleaves(KIND) || 2 * s >= R ? make_int2(4 * s, 4 * s + 2) : make_int2(2 * s, R + 2 * s); };
        const int2 x = slot(t), y = slot(t + G);
        return {x.x, y.x, x.y, y.y};
    } else {
        if (KIND == kHalves && 4 * t < R) return {4 * t, 4 * t + 2, R + 4 * t, R + 4 * t + 2};
        return {8 * t, 8 * t + 2, 8 * t + 4, 8 * t + 6};
    }
}

// A thread's eight channels as they were loaded, so that several rows are in flight without their fp32 copies
template <typename T, int W>
struct Row {
    float x[8];
    __device__ __forceinline__ void load(const T *p, int d, int t, int G, Runs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = t + G * i < d ? get(p + t + G * i) : 0.f;
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    __device__ __forceinline__ void unpack(float *y) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
    }
};
template <>
struct Row<bf16, 4> {
    uint2 a, b;
    __device__ __forceinline__ void clear() { a = b = make_uint2(0, 0); }
    __device__ __forceinline__ void load(const bf16 *p, int d, int, int, Runs r) {
        clear();
        if (r.a < d) {
            a = *reinterpret_cast<const uint2 *>(p + r.a);
            b = *reinterpret_cast<const uint2 *>(p + r.b);
        }
    }
    __device__ __forceinline__ void unpack(float *y) const {
        const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = __uint_as_float(w[i] << 16);
            y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Row<float, 4> {
    float4 a, b;
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float *p, int d, int, int, Runs r) {
        clear();
        if (r.a < d) {
            a = *reinterpret_cast<const float4 *>(p + r.a);
            b = *reinterpret_cast<const float4 *>(p + r.b);
        }
    }
    __device__ __forceinline__ void unpack(float *y) const {
        y[0] = a.x; y[1] = a.y; y[2] = a.z; y[3] = a.w;
        y[4] = b.x; y[5] = b.y; y[6] = b.z; y[7] = b.w;
    }
};
template <>
struct Row<bf16, 2> : Row<bf16, 4> {
    __device__ __forceinline__ void load(const bf16 *p, int d, int, int, Runs r) {
        clear();
        if (r.a < d) {
            a.x = *reinterpret_cast<const uint32_t *>(p + r.a);
            b.x = *reinterpret_cast<const uint32_t *>(p + r.b);
        }
        if (r.a2 < d) {
            a.y = *reinterpret_cast<const uint32_t *>(p + r.a2);
            b.y = *reinterpret_cast<const uint32_t *>(p + r.b2);
        }
    }
};
template <>
struct Row<float, 2> : Row<float, 4> {
    __device__ __forceinline__ void load(const float *p, int d, int, int, Runs r) {
        clear();
        auto at = [&](int c) { return *reinterpret_cast<const float2 *>(p + c); };
        if (r.a < d) {
            const float2 x = at(r.a), y = at(r.b);
            a.x = x.x; a.y = x.y; b.x = y.x; b.y = y.y;
        }
        if (r.a2 < d) {
            const float2 x = at(r.a2), y = at(r.b2);
            a.z = x.x; a.w = x.y; b.z = y.x; b.w = y.y;
        }
    }
};
template <int W>
__device__ __forceinline__ void store_row(float *p, const float *x, int d, int t, int G, Runs r) {
    if constexpr (W == 4) {
        if (r.a < d) {
            *reinterpret_cast<float4 *>(p + r.a) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4 *>(p + r.b) = make_float4(x[4], x[5], x[6], x[7]);
        }
    } else if constexpr (W == 2) {
        auto put = [&](int c, float lo, float hi) { *reinterpret_cast<float2 *>(p + c) = make_float2(lo, hi); };
        if (r.a < d) {
            put(r.a, x[0], x[1]);
            put(r.b, x[4], x[5]);
        }
        if (r.a2 < d) {
            put(r.a2, x[2], x[3]);
            put(r.b2, x[6], x[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t + G * i < d) p[t + G * i] = x[i];
    }
}
template <int W>
__device__ __forceinline__ void store_row(bf16 *p, const float *x, int d, int t, int G, Runs r) {
    if constexpr (W == 4) {
        if (r.a < d) {
            *reinterpret_cast<uint2 *>(p + r.a) = make_uint2(ptx::pack_bf16(x[0], x[1]), ptx::pack_bf16(x[2], x[3]));
            *reinterpret_cast<uint2 *>(p + r.b) = make_uint2(ptx::pack_bf16(x[4], x[5]), ptx::pack_bf16(x[6], x[7]));
        }
    } else if constexpr (W == 2) {
        auto put = [&](int c, float lo, float hi) { *reinterpret_cast<uint32_t *>(p + c) = ptx::pack_bf16(lo, hi); };
        if (r.a < d) {
            put(r.a, x[0], x[1]);
            put(r.b, x[4], x[5]);
        }
        if (r.a2 < d) {
            put(r.a2, x[2], x[3]);
            put(r.b2, x[6], x[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t + G * i < d) p[t + G * i] = __float2bfloat16_rn(x[i]);
    }
}
__device__ __forceinline__ float group_sum(float x, int G) {
    for (int o = G >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The row x turned by its token's angles, cs the (cos, sin) of this thread's four pairs or, by single channels, of each of its
// eight channels' pairs; sign = -1: back. stage: 2 R floats of this group (single channels). The whole warp calls it.
template <Kind KIND>
__device__ __forceinline__ void turn(float *x, const float2 *cs, int R, bool interleaved, float sign, int t, int G, float *stage) {
    if constexpr (KIND != kSingle) {  // threads without pairs have the angle 0
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float &a = interleaves(KIND) ? x[2 * i] : x[i], &b = interleaves(KIND) ? x[2 * i + 1] : x[4 + i];
            const float s = sign * cs[i].y, y = a * cs[i].x - b * s;
            b = fmaf(b, cs[i].x, a * s);
            a = y;
        }
    } else {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t + G * i < 2 * R) stage[t + G * i] = x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = t + G * i;
            if (c < 2 * R) {
                const bool low = interleaved ? (c & 1) == 0 : c < R;
                const float other = stage[interleaved ? c ^ 1 : low ? c + R : c - R];
                x[i] = fmaf(low ? -other : other, sign * cs[i].y, x[i] * cs[i].x);
            }
        }
    }
}

__device__ __forceinline__ int64_t position(const QkNormArgs &p, int64_t t) {
    return p.wide_positions ? static_cast<const int64_t *>(p.positions)[t] : static_cast<const int32_t *>(p.positions)[t];
}

// Rows of a group that are in flight at once
template <bool BWD>
constexpr int kBatch = BWD ? 2 : 4;

// A CTA's warps take kThreads / 32 / share tokens at a time, share of them the heads of one; every
// gridDim.x-th of such blocks of tokens. Dynamic shared memory (single channels): the groups' stages.
template <typename T, Kind KIND, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? 3 : 4) qk_norm_kernel(const QkNormArgs p, int G, int share) {
    extern __shared__ __align__(16) float stages[];
    __shared__ __align__(16) float weight[2][kMaxD];
    __shared__ uint64_t fraction[kMaxD / 2];
    constexpr int W = width(KIND), NB = kBatch<BWD>, NA = W > 1 ? 4 : 8;
    if constexpr (BWD) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int R = p.n_freqs, tid = threadIdx.x, warp = tid >> 5, t = tid & (G - 1);
    const int per_warp = 32 / G, first = (warp % share) * per_warp + (tid & 31) / G, stride = share * per_warp;  // heads
    const Runs run = runs<KIND>(t, R, G);
    float *stage = stages + tid / G * 2 * R;
    for (int i = tid; i < kMaxD; i += kThreads) {
        weight[0][i] = i < p.d ? p.weight[0][i] : 0.f;
        weight[1][i] = i < p.d ? p.weight[1][i] : 0.f;
    }
    for (int i = tid; i < R; i += kThreads) fraction[i] = turn_fraction(p.freqs[i]);
    __syncthreads();
    float dw[2][8];
    if constexpr (BWD)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[n][i] = 0.f;
    const float inv_d = 1.f / p.d;
    const int tokens = kThreads / 32 / share;
    for (int64_t tok = (int64_t)blockIdx.x * tokens + warp / share; tok < p.n_tok; tok += (int64_t)gridDim.x * tokens) {
        float2 cs[NA];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int heads = p.heads[which];
            const T *x_at = static_cast<const T *>(p.x[which]) + tok * p.stride[which];  // offsets of heads fit 32 bits
            const T *u_at = BWD ? static_cast<const T *>(p.dy[which]) + tok * p.dy_stride[which] : nullptr;
            T *y_at = static_cast<T *>(p.y[which]) + tok * heads * p.d;
            Row<T, W> x_row[NB], u_row[BWD ? NB : 1];
            auto fetch = [&](int n, int h) {
                if (h < heads) {
                    x_row[n].load(x_at + h * p.d, p.d, t, G, run);
                    if constexpr (BWD) u_row[n].load(u_at + h * p.d, p.d, t, G, run);
                } else {
                    x_row[n].clear();
                    if constexpr (BWD) u_row[n].clear();
                }
            };
#pragma unroll
            for (int n = 0; n < NB; ++n) fetch(n, first + n * stride);
            if (which == 0) {  // while the first rows are under way
                const uint64_t at = R > 0 ? (uint64_t)position(p, tok) : 0;
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    const int c = t + G * i;
                    const int pair = KIND == kHalves2        ? 2 * (t + (i >> 1) * G) + (i & 1)
                                     : KIND == kInterleaved2 ? 2 * (t + (i & 1) * G) + (i >> 1)
                                     : W == 4                ? 4 * t + i
                                     : p.interleaved         ? c >> 1
                                     : c < R                 ? c
                                                             : c - R;
                    cs[i] = cos_sin((W > 1 ? pair < R : c < 2 * R) ? fraction[pair] * at : 0);
                }
            }
            float w[8];
            if constexpr (W == 2) {
                const int at[4] = {run.a, run.a2, run.b, run.b2};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 x = *reinterpret_cast<const float2 *>(&weight[which][min(at[i], kMaxD - 2)]);
                    w[2 * i] = x.x;
                    w[2 * i + 1] = x.y;
                }
            } else if constexpr (W == 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&weight[which][min(run.a, kMaxD - 4)]);
                const float4 b = *reinterpret_cast<const float4 *>(&weight[which][min(run.b, kMaxD - 4)]);
                w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
                w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = weight[which][t + G * i];
            }
            // as many rounds for all groups of a warp: its threads meet in the sums
#pragma unroll 1
            for (int h0 = first; h0 - (tid & 31) / G < heads; h0 += NB * stride) {
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const int h = h0 + n * stride;
                    const bool live = h < heads;
                    float x[8], u[8];
                    x_row[n].unpack(x);
                    if constexpr (BWD) u_row[n].unpack(u);
                    fetch(n, h + NB * stride);  // on its way as soon as its registers are free
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
                    ss = group_sum(ss, G);
                    const float c = rsqrtf(ss * inv_d + p.eps);  // 2^-22 at most
                    if constexpr (!BWD) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] *= c * w[i];
                        turn<KIND>(x, cs, R, p.interleaved, 1.f, t, G, stage);
                        if (live) store_row<W>(y_at + h * p.d, x, p.d, t, G, run);
                    } else {
                        turn<KIND>(u, cs, R, p.interleaved, -1.f, t, G, stage);
                        float tn = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x[i] *= c;
                            dw[which][i] = fmaf(u[i], x[i], dw[which][i]);
                            u[i] *= w[i];
                            tn = fmaf(u[i], x[i], tn);
                        }
                        tn = group_sum(tn, G) * inv_d;
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] = c * (u[i] - x[i] * tn);
                        if (live) store_row<W>(y_at + h * p.d, u, p.d, t, G, run);
                    }
                }
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
                const int c = W > 1 ? (i < 2 ? run.a : i < 4 ? run.a2 : i < 6 ? run.b : run.b2) + (i & 1) : t + G * i;
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

// dw[n][c] = the sum of the partial rows, 32 channels a CTA, the rows dealt out to its warps
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) qk_norm_sum_kernel(const float *partial, int rows, int d, float *dq, float *dk) {
    const int n = blockIdx.y, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, part = threadIdx.x >> 5;
    __shared__ float sum[kSumThreads / 32][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float x = 0.f;
    if (c < d) {
        const float *at = partial + (int64_t)n * rows * d + c;
#pragma unroll 8
        for (int i = part; i < rows; i += kSumThreads / 32) x += at[(int64_t)i * d];
    }
    sum[part][lane] = x;
    __syncthreads();
    if (part == 0 && c < d) {
        x = 0.f;
#pragma unroll
        for (int i = 0; i < kSumThreads / 32; ++i) x += sum[i][lane];
        (n ? dk : dq)[c] = x;
    }
}

constexpr int kBlocks = 152 * 4, kBwdBlocks = 152 * 3;

// The most channels of a row at once that lengths, halves and addresses allow
template <typename T>
int load_width(const QkNormArgs &p, bool bwd) {
    uintptr_t all = 0;
    for (int i = 0; i < 2; ++i)
        all |= (uintptr_t)p.x[i] | (uintptr_t)p.y[i] | (bwd ? (uintptr_t)p.dy[i] | (uintptr_t)p.dy_stride[i] * sizeof(T) : 0) |
               (uintptr_t)p.stride[i] * sizeof(T);
    if (p.d % 8 == 0 && p.n_freqs % 4 == 0 && all % (4 * sizeof(T)) == 0) return 4;
    return p.d % 4 == 0 && (p.interleaved || p.n_freqs % 2 == 0) && all % (2 * sizeof(T)) == 0 ? 2 : 1;
}

template <typename T, bool BWD>
cudaError_t run(const QkNormArgs &p, cudaStream_t stream) {
    int G = 1;
    while (8 * G < p.d) G *= 2;
    const int warps = kThreads / 32, heads = std::max(p.heads[0], p.heads[1]);
    // A token to a warp, which forms its angles; with too few tokens for the warps of all SMs to several, as far
    // as there are heads (backward, whose rows take longer, with less than four each)
    int share = 1;
    while (share < warps && p.n_tok * share < (BWD ? 4 * kBwdBlocks : kBlocks) * warps && share * (32 / G) < heads) share *= 2;
    const int64_t blocks = (p.n_tok * share + warps - 1) / warps;
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, BWD ? kBwdBlocks : kBlocks);
    const int w = load_width<T>(p, BWD);
    const size_t smem = w > 1 ? 0 : (size_t)kThreads / G * 2 * p.n_freqs * 4;
    if (grid > 0) {
        auto kernel = w == 1          ? qk_norm_kernel<T, kSingle, BWD>
                      : p.interleaved ? w == 4 ? qk_norm_kernel<T, kInterleaved, BWD> : qk_norm_kernel<T, kInterleaved2, BWD>
                      : w == 4        ? qk_norm_kernel<T, kHalves, BWD>
                                      : qk_norm_kernel<T, kHalves2, BWD>;
        kernel<<<grid, kThreads, smem, stream>>>(p, G, share);
        count_launches(1);
    }
    if (BWD) {
        // launched early: it waits for the partial rows on the device
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((p.d + 31) / 32, 2);
        cfg.blockDim = dim3(kSumThreads);
        cfg.stream = stream;
        cfg.attrs = &attr;
        cfg.numAttrs = grid > 0 ? 1 : 0;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, qk_norm_sum_kernel, (const float *)p.partial, (int)grid, (int)p.d, p.dw[0], p.dw[1]);
        if (e != cudaSuccess) return e;
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
