// kda_norm.cu -- the norms around a recurrence block, forward and backward.
//
// Residual norm, a row of d channels (before a block; x is the previous block's output):
//   r = residual + scale x,   y = w r c,   c = (mean r^2 + eps)^-1/2
//   backward, with n = r c, t = w dy:  dr' = dr + c (t - n mean(t n));  dresidual = dr',
//   dx = scale dr', dscale = sum over rows of x dr', dw = sum over rows of dy n
// Gated norm, a row of d channels of one (token, head) (after the recurrence):
//   y = w n act(z),  n = x c;   backward with t = w act(z) dy:
//   dx = c (t - n mean(t n)),  dz = dy w n act'(z),  dw = sum over rows of dy n act(z)
// Sums and statistics are fp32. All are bound by HBM: every input is read once, kept in
// registers across the row's reduction, every output written once. The sums over rows go to
// one partial row per CTA (group), added up in a fixed order by a second kernel: the same
// call gives the same bits.
// bf16, of a plain copy's bandwidth: residual norm forward, 32K rows of 4096 or 8192 channels, 1.0
// and 0.93 (155 and 339 us); its backward pass 0.90 (32K x 4096, 262 us); gated norm forward 0.96
// (64K tokens x 32 heads x 128, 248 us), backward 0.83 (8191 tokens x 32 x 128, 59 us, of them 5 the
// sum over partial rows; 64K tokens 0.97).
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

#include "kda_internal.h"
#include "kda_ptx.h"

namespace kda {
namespace {

using bf16 = __nv_bfloat16;

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
    uint4 a;
    a.x = ptx::pack_bf16(x[0], x[1]);
    a.y = ptx::pack_bf16(x[2], x[3]);
    a.z = ptx::pack_bf16(x[4], x[5]);
    a.w = ptx::pack_bf16(x[6], x[7]);
    *reinterpret_cast<uint4 *>(p) = a;
}

// A group of G threads holds a row of d channels, 8 NV of them per thread: with VEC thread
// t the 8-channel runs 8 (t + G i), otherwise the channels t + G i one by one.
template <int NV, bool VEC, typename T>
__device__ __forceinline__ void load_row(const T *p, int d, int t, int G, float *x) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if constexpr (VEC) {
            const int c = 8 * (t + G * i);
            if (c < d) load8(p + c, x + 8 * i);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) x[8 * i + j] = 0.f;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = t + G * (8 * i + j);
                x[8 * i + j] = c < d ? get(p + c) : 0.f;
            }
        }
    }
}
template <int NV, bool VEC, typename T>
__device__ __forceinline__ void store_row(T *p, int d, int t, int G, const float *x) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if constexpr (VEC) {
            const int c = 8 * (t + G * i);
            if (c < d) store8(p + c, x + 8 * i);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = t + G * (8 * i + j);
                if (c < d) put(p + c, x[8 * i + j]);
            }
        }
    }
}

// A thread's 8 NV channels of a row as they were loaded: unpacked to floats only at use, so
// that several rows' worth of loads can be in flight without their fp32 copies' registers.
template <typename T, int NV, bool VEC>
struct Held {
    float x[8 * NV];
    __device__ __forceinline__ void load(const T *p, int d, int t, int G) { load_row<NV, VEC>(p, d, t, G, x); }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8 * NV; ++i) x[i] = 0.f;
    }
    __device__ __forceinline__ void put_run(int run, uint4 a) {
        x[4 * run] = __uint_as_float(a.x);
        x[4 * run + 1] = __uint_as_float(a.y);
        x[4 * run + 2] = __uint_as_float(a.z);
        x[4 * run + 3] = __uint_as_float(a.w);
    }
    __device__ __forceinline__ float get(int i) const { return x[i]; }
};
template <int NV>
struct Held<bf16, NV, true> {
    uint32_t w[4 * NV];
    __device__ __forceinline__ void load(const bf16 *p, int d, int t, int G) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (t + G * i);
            uint4 a = make_uint4(0, 0, 0, 0);
            if (c < d) a = *reinterpret_cast<const uint4 *>(p + c);
            w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void put_run(int, uint4 a) { w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; }
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};

// Rows ahead of their use. A thread copies its 8 channels of N tensors' rows to slots of its own in
// shared memory and reads them back itself: the next row is in flight, without registers for it
// and without a barrier, while this one's sums are formed and its results written.
template <typename T, int N, int THREADS>
struct Ahead {
    static constexpr int kRuns = sizeof(T) / 2, kBytes = N * kRuns * THREADS * 16;  // 16-byte runs
    char *slots;
    __device__ __forceinline__ explicit Ahead(char *smem) : slots(smem + threadIdx.x * 16) {}
    __device__ __forceinline__ char *at(int n, int run) const { return slots + (n * kRuns + run) * (THREADS * 16); }
    // channels 8 t .. of the row at p, zeros from d on
    __device__ __forceinline__ void fetch(int n, const T *p, int d, int t) const {
        const bool in = 8 * t < d;
#pragma unroll
        for (int run = 0; run < kRuns; ++run)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(at(n, run))),
                         "l"(in ? p + 8 * t + run * (16 / sizeof(T)) : p), "r"(in ? 16 : 0) : "memory");
    }
    __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
    __device__ __forceinline__ void read(int n, Held<T, 1, true> &h) const {
#pragma unroll
        for (int run = 0; run < kRuns; ++run) {
            const uint4 a = *reinterpret_cast<const uint4 *>(at(n, run));
            h.put_run(run, a);
        }
    }
};

// Sum over the G threads (G = 32 WPR) of a group; every thread gets it. `buf` holds WPR
// floats per group and alternates between two halves so that one barrier per sum suffices.
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
template <int WPR>
__device__ __forceinline__ float group_sum(float x, float *buf, int group) {
    x = warp_sum(x);
    if constexpr (WPR > 1) {
        const int w = (threadIdx.x >> 5) % WPR;
        if ((threadIdx.x & 31) == 0) buf[group * WPR + w] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) x += buf[group * WPR + i];
    }
    return x;
}

// two sums at once, one barrier; `buf` (WPR pairs per group) alternates between two halves
template <int WPR>
__device__ __forceinline__ float2 group_sum2(float2 x, float2 *buf, int group) {
    x.x = warp_sum(x.x);
    x.y = warp_sum(x.y);
    if constexpr (WPR > 1) {
        const int w = (threadIdx.x >> 5) % WPR;
        if ((threadIdx.x & 31) == 0) buf[group * WPR + w] = x;
        __syncthreads();
        const int l = threadIdx.x & 31;
        x = l < WPR ? buf[group * WPR + l] : make_float2(0.f, 0.f);
#pragma unroll
        for (int o = WPR / 2; o > 0; o >>= 1) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
            x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
        }
        x.x = __shfl_sync(0xffffffffu, x.x, 0);
        x.y = __shfl_sync(0xffffffffu, x.y, 0);
    }
    return x;
}

template <int WPR>
struct Rows {
    static constexpr int kWarps = WPR < 8 ? 8 : WPR;
    static constexpr int kThreads = 32 * kWarps, kGroups = kWarps / WPR, G = 32 * WPR;
};

template <typename T, int WPR, int NV, bool VEC>
__global__ void __launch_bounds__(Rows<WPR>::kThreads)
    residual_norm_fwd_kernel(const ResidualNormArgs p) {
    using L = Rows<WPR>;
    __shared__ float buf[L::kWarps];
    const int group = threadIdx.x / L::G, t = threadIdx.x % L::G;
    const int64_t row = (int64_t)blockIdx.x * L::kGroups + group;
    const bool live = row < p.n_rows;
    float r[8 * NV], w[8 * NV];
#pragma unroll
    for (int i = 0; i < 8 * NV; ++i) r[i] = 0.f;
    if (live) {
        Held<T, NV, VEC> x, res;
        x.load(static_cast<const T *>(p.x) + row * p.x_stride, p.d, t, L::G);
        if (p.residual) res.load(static_cast<const T *>(p.residual) + row * p.residual_stride, p.d, t, L::G);
        else res.clear();
        load_row<NV, VEC>(p.weight, p.d, t, L::G, w);
        if (p.scale) {
            load_row<NV, VEC>(p.scale, p.d, t, L::G, r);
#pragma unroll
            for (int i = 0; i < 8 * NV; ++i) r[i] = fmaf(r[i], x.get(i), res.get(i));
        } else {
#pragma unroll
            for (int i = 0; i < 8 * NV; ++i) r[i] = x.get(i) + res.get(i);
        }
        if (p.r) store_row<NV, VEC>(static_cast<T *>(p.r) + row * p.d, p.d, t, L::G, r);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * NV; ++i) s = fmaf(r[i], r[i], s);
    s = group_sum<WPR>(s, buf, group);
    if (!live) return;
    const float c = 1.f / sqrtf(s / p.d + p.eps);
#pragma unroll
    for (int i = 0; i < 8 * NV; ++i) w[i] *= r[i] * c;
    store_row<NV, VEC>(static_cast<T *>(p.y) + row * p.d, p.d, t, L::G, w);
}

// Each group walks over rows first, first + step, ...; its sums of dw (and dscale) go to
// row `blockIdx.x * kGroups + group` of the partials. The next row is copied ahead from the moment
// that this one is in registers (32768 x 4096, bf16: 264 us; without it 302; two rows ahead 285).
template <typename T, int WPR, int NV, bool VEC, bool SCALE>
__global__ void __launch_bounds__(Rows<WPR>::kThreads, NV == 1 ? 1024 / Rows<WPR>::kThreads : 1)
    residual_norm_bwd_kernel(const ResidualNormArgs p, int64_t rounds) {
    using L = Rows<WPR>;
    __shared__ float2 buf[2][L::kWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int group = threadIdx.x / L::G, t = threadIdx.x % L::G;
    const int64_t part = (int64_t)blockIdx.x * L::kGroups + group, step = (int64_t)gridDim.x * L::kGroups;
    const float inv_d = 1.f / p.d;
    // weight and scale wait in shared memory (up to 8192 channels, else they are reloaded
    // through the cache): 16 registers fewer, which two CTAs of 512 threads need
    extern __shared__ __align__(16) float params[];
    constexpr bool AHEAD = VEC && NV == 1;
    const Ahead<T, SCALE ? 4 : 3, L::kThreads> ahead(reinterpret_cast<char *>(params + (SCALE ? 2 : 1) * p.d));
    auto fetch = [&](int64_t i) {
        const int64_t row = part + i * step;
        if (row < p.n_rows) {
            ahead.fetch(0, static_cast<const T *>(p.r) + row * p.r_stride, p.d, t);
            ahead.fetch(1, static_cast<const T *>(p.dy) + row * p.dy_stride, p.d, t);
            if (p.dr) ahead.fetch(2, static_cast<const T *>(p.dr) + row * p.dr_stride, p.d, t);
            if constexpr (SCALE) ahead.fetch(3, static_cast<const T *>(p.x) + row * p.x_stride, p.d, t);
        }
    };
    if constexpr (AHEAD) fetch(0);
    const float *weight = p.weight, *scale = p.scale;
    if constexpr (NV == 1) {
        for (int i = threadIdx.x; i < p.d; i += L::kThreads) {
            params[i] = p.weight[i];
            if constexpr (SCALE) params[p.d + i] = p.scale[i];
        }
        weight = params;
        scale = params + p.d;
        __syncthreads();
    }
    float dw[8 * NV], ds[SCALE ? 8 * NV : 1];
#pragma unroll
    for (int i = 0; i < 8 * NV; ++i) dw[i] = 0.f;
    if constexpr (SCALE)
#pragma unroll
        for (int i = 0; i < 8 * NV; ++i) ds[i] = 0.f;
    for (int64_t i0 = 0; i0 < rounds; ++i0) {
        const int64_t row = part + i0 * step;
        const bool live = row < p.n_rows;
        Held<T, NV, VEC> r, dy, dr;
        [[maybe_unused]] Held<T, NV, VEC> x;
        r.clear();
        dy.clear();
        dr.clear();
        if constexpr (AHEAD) {
            ahead.wait();
            if (live) {
                ahead.read(0, r);
                ahead.read(1, dy);
                if (p.dr) ahead.read(2, dr);
                if constexpr (SCALE) ahead.read(3, x);
            }
        } else if (live) {
            r.load(static_cast<const T *>(p.r) + row * p.r_stride, p.d, t, L::G);
            dy.load(static_cast<const T *>(p.dy) + row * p.dy_stride, p.d, t, L::G);
            if (p.dr) dr.load(static_cast<const T *>(p.dr) + row * p.dr_stride, p.d, t, L::G);
            if constexpr (SCALE) x.load(static_cast<const T *>(p.x) + row * p.x_stride, p.d, t, L::G);
        }
        float2 sum = make_float2(0.f, 0.f);  // r^2 and w dy r
        float w[8 * NV];
        load_row<NV, VEC>(weight, p.d, t, L::G, w);
#pragma unroll
        for (int i = 0; i < 8 * NV; ++i) {
            sum.x = fmaf(r.get(i), r.get(i), sum.x);
            sum.y = fmaf(w[i] * dy.get(i), r.get(i), sum.y);
        }
        sum = group_sum2<WPR>(sum, buf[i0 & 1], group);
        if constexpr (AHEAD) fetch(i0 + 1);  // this row is in registers
        if (!live) continue;
        const float c = 1.f / sqrtf(fmaf(sum.x, inv_d, p.eps)), m = sum.y * c * c * inv_d;
        float g[8 * NV];
        load_row<NV, VEC>(weight, p.d, t, L::G, w);
#pragma unroll
        for (int i = 0; i < 8 * NV; ++i) {
            g[i] = fmaf(c, fmaf(w[i], dy.get(i), -r.get(i) * m), dr.get(i));
            dw[i] = fmaf(dy.get(i) * c, r.get(i), dw[i]);
        }
        store_row<NV, VEC>(static_cast<T *>(p.dresidual) + row * p.d, p.d, t, L::G, g);
        if constexpr (SCALE) {
            load_row<NV, VEC>(scale, p.d, t, L::G, w);
#pragma unroll
            for (int i = 0; i < 8 * NV; ++i) {
                ds[i] = fmaf(x.get(i), g[i], ds[i]);
                g[i] *= w[i];
            }
            store_row<NV, VEC>(static_cast<T *>(p.dx) + row * p.d, p.d, t, L::G, g);
        }
    }
    store_row<NV, VEC>(p.partial + part * p.d, p.d, t, L::G, dw);
    if constexpr (SCALE) store_row<NV, VEC>(p.partial + (step + part) * p.d, p.d, t, L::G, ds);
}

// out[c] = sum over the parts of partial[part][c], in a fixed order; blockIdx.y chooses the sum
__global__ void __launch_bounds__(1024)
    sum_parts_kernel(const float *__restrict__ partial, int parts, int d, float *__restrict__ out0,
                     float *__restrict__ out1) {
    __shared__ float s[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), l = threadIdx.x >> 5;
    const float *src = partial + (int64_t)blockIdx.y * parts * d;
    float x = 0.f;
    if (c < d)
#pragma unroll 8
        for (int i = l; i < parts; i += 32) x += src[(int64_t)i * d + c];
    s[l][threadIdx.x & 31] = x;
    __syncthreads();
    if (blockIdx.x * 32 + l < d) {  // warp l adds up column l
        x = warp_sum(s[threadIdx.x & 31][l]);
        if ((threadIdx.x & 31) == 0) (blockIdx.y ? out1 : out0)[blockIdx.x * 32 + l] = x;
    }
}

constexpr int kSMs = 152;

// launched while the kernel before it drains: the launch's latency, 2 us of 60, passes meanwhile
cudaError_t sum_parts(const float *partial, int parts, int d, float *out0, float *out1, cudaStream_t stream) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((d + 31) / 32, out1 ? 2 : 1);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sum_parts_kernel, partial, parts, d, out0, out1);
}

// Warps to a row (a power of two) and 8-channel runs to a thread: one run up to 8192 channels, so
// that a row's loads are all in flight at once; beyond, a CTA has no more threads.
struct RowPlan { int wpr, nv; };
RowPlan row_plan(int d) {
    int wpr = 1;
    while (wpr < 32 && 256 * wpr < d) wpr *= 2;
    return {wpr, 256 * wpr >= d ? 1 : 512 * wpr >= d ? 2 : 4};
}
int plan_groups(const RowPlan &r) { return r.wpr < 8 ? 8 / r.wpr : 1; }
int64_t residual_bwd_grid(int64_t n_rows, int d) {
    const RowPlan r = row_plan(d);
    const int per_sm = r.nv > 1 ? 1 : r.wpr <= 8 ? 4 : 32 / r.wpr;
    return std::max<int64_t>(1, std::min<int64_t>((n_rows + plan_groups(r) - 1) / plan_groups(r), kSMs * per_sm));
}

template <typename T, int WPR, int NV, bool VEC>
cudaError_t residual_run(const ResidualNormArgs &p, bool bwd, cudaStream_t stream) {
    using L = Rows<WPR>;
    if (!bwd) {
        residual_norm_fwd_kernel<T, WPR, NV, VEC>
            <<<(unsigned)((p.n_rows + L::kGroups - 1) / L::kGroups), L::kThreads, 0, stream>>>(p);
        count_launches(1);
        return cudaGetLastError();
    }
    const int64_t grid = residual_bwd_grid(p.n_rows, p.d), parts = grid * L::kGroups;
    const int64_t rounds = (p.n_rows + parts - 1) / parts;
    constexpr int most_d = 256 * WPR;  // channels of this instance where it keeps the parameters in shared memory
    const int ahead = VEC && NV == 1 ? p.scale ? Ahead<T, 4, L::kThreads>::kBytes
                                              : Ahead<T, 3, L::kThreads>::kBytes : 0;
    const int per_d = NV == 1 ? p.scale ? 8 : 4 : 0, smem = p.d * per_d + ahead, most = most_d * per_d + ahead;
    auto kernel = p.scale ? residual_norm_bwd_kernel<T, WPR, NV, VEC, true> : residual_norm_bwd_kernel<T, WPR, NV, VEC, false>;
    if (most + (int)sizeof(float2) * 2 * L::kWarps > 48 * 1024) {  // with the static buffers
        const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), most);
        if (e != cudaSuccess) return e;
    }
    kernel<<<(unsigned)grid, L::kThreads, smem, stream>>>(p, rounds);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = sum_parts(p.partial, (int)parts, p.d, p.dw, p.scale ? p.dscale : nullptr, stream);
    if (e != cudaSuccess) return e;
    count_launches(2);
    return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t residual_pick(const ResidualNormArgs &p, bool bwd, cudaStream_t s) {
    const RowPlan r = row_plan(p.d);
    if (r.nv == 4) return residual_run<T, 32, 4, VEC>(p, bwd, s);
    if (r.nv == 2) return residual_run<T, 32, 2, VEC>(p, bwd, s);
    switch (r.wpr) {
        case 1: return residual_run<T, 1, 1, VEC>(p, bwd, s);
        case 2: return residual_run<T, 2, 1, VEC>(p, bwd, s);
        case 4: return residual_run<T, 4, 1, VEC>(p, bwd, s);
        case 8: return residual_run<T, 8, 1, VEC>(p, bwd, s);
        case 16: return residual_run<T, 16, 1, VEC>(p, bwd, s);
        default: return residual_run<T, 32, 1, VEC>(p, bwd, s);
    }
}

bool vec_ok(const void *p, int64_t stride, int es) {
    return ((uintptr_t)p & 15u) == 0 && (stride * es) % 16 == 0;
}

// ---------------------------------------------------------------- gated norm

// act(z): silu when SILU, else the sigmoid. FAST (bf16 tensors): the hardware's exponential and
// quotient, within a few units in 2^-22 of the sigmoid, far below the result's rounding to bf16;
// with the accurate forms the bf16 kernels are bound by instruction issue instead of HBM.
template <bool SILU, bool FAST>
__device__ __forceinline__ float act(float z) {
    const float s = FAST ? __fdividef(1.f, 1.f + __expf(-z)) : 1.f / (1.f + expf(-z));
    return SILU ? z * s : s;
}
// The sigmoid s and rest = 1 - s, of which act' is formed: s rest, or s (1 + z rest) for silu. rest is
// exp(-z) s: as a difference it has lost 1e-3 at z = 10 and everything at 17, where s rounds to 1.
// The bound takes an infinite exp(-z), where s is 0, out of that product.
template <bool FAST>
__device__ __forceinline__ void act_parts(float z, float &s, float &rest) {
    const float e = FAST ? __expf(-z) : expf(-z);
    s = FAST ? __fdividef(1.f, 1.f + e) : 1.f / (1.f + e);
    rest = fminf(e, FLT_MAX) * s;
}

// row / n_heads for row < 2^31 as a multiplication, (umulhi(row, m) + row) >> s: division by an
// invariant (Granlund and Montgomery, 1994)
struct HeadDiv { uint32_t m, s; };
HeadDiv head_div(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return {(uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1), s};
}
__device__ __forceinline__ uint32_t divide(uint32_t row, HeadDiv h) { return (__umulhi(row, h.m) + row) >> h.s; }

constexpr int kGatedThreads = 256;

// G threads (a power of two up to a warp) hold a row of d <= 8 G channels.
// A CTA walks over rows with the next one copied ahead; the grid is the CTAs that the SMs hold.
// 65536 x 32 x 128, bf16: 248 us with five an SM, 262 with four, 276 with six (more requests in
// flight than HBM orders well), 304 with six of which five are resident; a row a group and no
// loop 283.
constexpr int kGatedFwdCtas = 5;
template <typename T, int G, bool VEC, bool SILU>
__global__ void __launch_bounds__(kGatedThreads, kGatedFwdCtas)
    gated_norm_fwd_kernel(const GatedNormArgs p, const HeadDiv by) {
    const int t = threadIdx.x % G;
    constexpr int kGroups = kGatedThreads / G;
    const int64_t rows = p.n_tok * p.n_heads, step = (int64_t)gridDim.x * kGroups;
    extern __shared__ __align__(16) char slots[];
    const Ahead<T, 2, kGatedThreads> ahead(slots);
    Held<T, 1, VEC> hx, hz;
    // channel 0 of the row's head in x and gate
    auto heads = [&](int64_t row, auto use) {
        const uint32_t n = divide((uint32_t)row, by);
        const int64_t h = (int64_t)((uint32_t)row - n * p.n_heads) * p.d;
        use(static_cast<const T *>(p.x) + n * p.x_stride + h, static_cast<const T *>(p.gate) + n * p.gate_stride + h);
    };
    auto fetch = [&](int64_t row) {
        if (row < rows)
            heads(row, [&](const T *px, const T *pz) {
                ahead.fetch(0, px, p.d, t);
                ahead.fetch(1, pz, p.d, t);
            });
    };
    float w[8];
    load_row<1, VEC>(p.weight, p.d, t, G, w);
    int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / G;
    if constexpr (VEC) fetch(row);
    for (int64_t first = (int64_t)blockIdx.x * kGroups; first < rows; first += step, row += step) {
        const bool live = row < rows;
        hx.clear();
        hz.clear();
        if constexpr (VEC) {
            ahead.wait();
            if (live) {
                ahead.read(0, hx);
                ahead.read(1, hz);
            }
        } else if (live) {
            heads(row, [&](const T *px, const T *pz) {
                hx.load(px, p.d, t, G);
                hz.load(pz, p.d, t, G);
            });
        }
        float s = 0.f, x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = hx.get(i);
            s = fmaf(x[i], x[i], s);
        }
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if constexpr (VEC) fetch(row + step);  // this row is in registers
        if (!live) continue;
        const float c = 1.f / sqrtf(s / p.d + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = x[i] * c * w[i] * act<SILU, sizeof(T) == 2>(hz.get(i));
        }
        store_row<1, VEC>(static_cast<T *>(p.y) + row * p.d, p.d, t, G, x);
    }
}

template <typename T, int G, bool VEC, bool SILU>
__global__ void __launch_bounds__(kGatedThreads, 4)
    gated_norm_bwd_kernel(const GatedNormArgs p, const HeadDiv by, int64_t rounds) {
    constexpr int kGroups = kGatedThreads / G;
    __shared__ float sums[kGatedThreads / 32][8 * G];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = threadIdx.x % G;
    const int64_t rows = p.n_tok * p.n_heads, step = (int64_t)gridDim.x * kGroups;
    const float inv_d = 1.f / p.d;
    float w[8], dw[8];
    load_row<1, VEC>(p.weight, p.d, t, G, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = 0.f;
    extern __shared__ __align__(16) char slots[];
    const Ahead<T, 3, kGatedThreads> ahead(slots);
    const int64_t first = (int64_t)blockIdx.x * kGroups + threadIdx.x / G;
    Held<T, 1, VEC> x, z, dy;
    // channel 0 of the row's head in x, gate and dy
    auto heads = [&](int64_t row, auto use) {
        const uint32_t n = divide((uint32_t)row, by);
        const int64_t h = (int64_t)((uint32_t)row - n * p.n_heads) * p.d;
        use(static_cast<const T *>(p.x) + n * p.x_stride + h, static_cast<const T *>(p.gate) + n * p.gate_stride + h,
            static_cast<const T *>(p.dy) + n * p.dy_stride + h);
    };
    auto fetch = [&](int64_t i) {
        if (i * step + first < rows)
            heads(i * step + first, [&](const T *px, const T *pz, const T *py) {
                ahead.fetch(0, px, p.d, t);
                ahead.fetch(1, pz, p.d, t);
                ahead.fetch(2, py, p.d, t);
            });
    };
    if constexpr (VEC) fetch(0);
    for (int64_t i0 = 0; i0 < rounds; ++i0) {
        const int64_t row = i0 * step + first;
        const bool live = row < rows;
        x.clear();
        z.clear();
        dy.clear();
        if constexpr (VEC) {
            ahead.wait();
            if (live) {
                ahead.read(0, x);
                ahead.read(1, z);
                ahead.read(2, dy);
            }
        } else if (live) {
            heads(row, [&](const T *px, const T *pz, const T *py) {
                x.load(px, p.d, t, G);
                z.load(pz, p.d, t, G);
                dy.load(py, p.d, t, G);
            });
        }
        float xx = 0.f, tx = 0.f, a[8], b[8];  // act; 1 - s, for silu act'
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            act_parts<sizeof(T) == 2>(z.get(i), a[i], b[i]);
            if constexpr (SILU) {
                b[i] = a[i] * fmaf(z.get(i), b[i], 1.f);
                a[i] *= z.get(i);
            }
            xx = fmaf(x.get(i), x.get(i), xx);
            tx = fmaf(a[i] * dy.get(i) * w[i], x.get(i), tx);
        }
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) {
            xx += __shfl_xor_sync(0xffffffffu, xx, o);
            tx += __shfl_xor_sync(0xffffffffu, tx, o);
        }
        if constexpr (VEC) fetch(i0 + 1);  // this row is in registers
        if (!live) continue;
        const float c = 1.f / sqrtf(fmaf(xx, inv_d, p.eps)), m = tx * c * c * inv_d;
        float dx[8], dz[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = x.get(i) * c, da = dy.get(i) * a[i], wa = da * w[i];
            dx[i] = c * fmaf(-m, x.get(i), wa);
            dz[i] = (SILU ? w[i] * dy.get(i) : wa) * n * b[i];
            dw[i] = fmaf(da, n, dw[i]);
        }
        store_row<1, VEC>(static_cast<T *>(p.dx) + row * p.d, p.d, t, G, dx);
        store_row<1, VEC>(static_cast<T *>(p.dgate) + row * p.d, p.d, t, G, dz);
    }
    // the warp's groups, then the CTA's warps, in a fixed order
#pragma unroll
    for (int o = G; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
    if ((threadIdx.x & 31) < G)
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[threadIdx.x >> 5][VEC ? 8 * t + i : t + G * i] = dw[i];
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += kGatedThreads) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < kGatedThreads / 32; ++i) x += sums[i][c];
        p.partial[(int64_t)blockIdx.x * p.d + c] = x;
    }
}

int gated_group(int d) {
    int g = 4;
    while (8 * g < d) g *= 2;
    return g;
}
int64_t gated_bwd_grid(int64_t n_tok, int n_heads, int d) {
    const int per = kGatedThreads / gated_group(d);
    return std::max<int64_t>(1, std::min<int64_t>((n_tok * n_heads + per - 1) / per, kSMs * 4));
}

template <typename T, int G, bool VEC, bool SILU>
cudaError_t gated_run(const GatedNormArgs &p, bool bwd, cudaStream_t stream) {
    constexpr int kGroups = kGatedThreads / G;
    const int64_t rows = p.n_tok * p.n_heads;
    if (!bwd) {
        constexpr int smem = VEC ? Ahead<T, 2, kGatedThreads>::kBytes : 0;
        const int64_t grid = std::min<int64_t>((rows + kGroups - 1) / kGroups, kSMs * kGatedFwdCtas);
        gated_norm_fwd_kernel<T, G, VEC, SILU><<<(unsigned)grid, kGatedThreads, smem, stream>>>(p, head_div(p.n_heads));
        count_launches(1);
        return cudaGetLastError();
    }
    const int64_t grid = gated_bwd_grid(p.n_tok, p.n_heads, p.d), step = grid * kGroups;
    constexpr int smem = VEC ? Ahead<T, 3, kGatedThreads>::kBytes : 0;
    static_assert(smem + kGatedThreads * 16 <= 48 * 1024, "needs no attribute");
    gated_norm_bwd_kernel<T, G, VEC, SILU><<<(unsigned)grid, kGatedThreads, smem, stream>>>(p, head_div(p.n_heads), (rows + step - 1) / step);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = sum_parts(p.partial, (int)grid, p.d, p.dw, nullptr, stream);
    if (e != cudaSuccess) return e;
    count_launches(2);
    return cudaGetLastError();
}
template <typename T, bool VEC, bool SILU>
cudaError_t gated_pick(const GatedNormArgs &p, bool bwd, cudaStream_t s) {
    switch (gated_group(p.d)) {
        case 4: return gated_run<T, 4, VEC, SILU>(p, bwd, s);
        case 8: return gated_run<T, 8, VEC, SILU>(p, bwd, s);
        case 16: return gated_run<T, 16, VEC, SILU>(p, bwd, s);
        default: return gated_run<T, 32, VEC, SILU>(p, bwd, s);
    }
}
template <typename T>
cudaError_t gated(const GatedNormArgs &p, bool bwd, cudaStream_t s) {
    const int es = sizeof(T);
    bool vec = p.d % 8 == 0 && vec_ok(p.x, p.x_stride, es) && vec_ok(p.gate, p.gate_stride, es) &&
               vec_ok(p.weight, 0, 4);
    if (bwd) vec = vec && vec_ok(p.dy, p.dy_stride, es) && vec_ok(p.dx, 0, es) && vec_ok(p.dgate, 0, es);
    else vec = vec && vec_ok(p.y, 0, es);
    if (vec) return p.silu ? gated_pick<T, true, true>(p, bwd, s) : gated_pick<T, true, false>(p, bwd, s);
    return p.silu ? gated_pick<T, false, true>(p, bwd, s) : gated_pick<T, false, false>(p, bwd, s);
}

template <typename T>
cudaError_t residual(const ResidualNormArgs &p, bool bwd, cudaStream_t s) {
    const int es = sizeof(T);
    bool vec = p.d % 8 == 0 && vec_ok(p.weight, 0, 4) && vec_ok(p.scale, 0, 4) && vec_ok(p.x, p.x_stride, es);
    if (bwd)
        vec = vec && vec_ok(p.r, p.r_stride, es) && vec_ok(p.dy, p.dy_stride, es) && vec_ok(p.dr, p.dr_stride, es) &&
              vec_ok(p.dx, 0, es) && vec_ok(p.dresidual, 0, es);
    else
        vec = vec && vec_ok(p.residual, p.residual_stride, es) && vec_ok(p.r, 0, es) && vec_ok(p.y, 0, es);
    return vec ? residual_pick<T, true>(p, bwd, s) : residual_pick<T, false>(p, bwd, s);
}

}  // namespace

size_t residual_norm_workspace_bytes(int64_t n_rows, int32_t d, bool scale) {
    const RowPlan r = row_plan(d);
    return (size_t)residual_bwd_grid(n_rows, d) * plan_groups(r) * d * 4 * (scale ? 2 : 1);
}
size_t gated_norm_workspace_bytes(int64_t n_tok, int32_t n_heads, int32_t d) {
    return (size_t)gated_bwd_grid(n_tok, n_heads, d) * d * 4;
}
cudaError_t launch_residual_norm(const ResidualNormArgs &p, bool bwd, cudaStream_t s) {
    return p.bf16 ? residual<bf16>(p, bwd, s) : residual<float>(p, bwd, s);
}
cudaError_t launch_gated_norm(const GatedNormArgs &p, bool bwd, cudaStream_t s) {
    return p.bf16 ? gated<bf16>(p, bwd, s) : gated<float>(p, bwd, s);
}

}  // namespace kda
