// Shared by the tensor-core kernels of linear attention with one decay per head (bf16 inputs):
// segments, tiles, gates and the walk over a segment that carries the state. Internal.
//
// A tile is 64 tokens of one head in column halves of 64 channels, each 64 rows of 128 bytes in the
// 128-byte swizzle of tensor copies, which tcgen05 reads K-major or MN-major as it stands. Operands
// that are not bf16 inputs are sums of two bf16 planes (2^-18 of relative rounding).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_dla.h"

namespace kda {
namespace dla {

constexpr int C = 64;            // tokens of a tile
constexpr int kHalf = C * 128;   // bytes of a tile's 64 channels
constexpr long long kWaitLimit = 4000000000LL;  // SM cycles, about two seconds

static __device__ unsigned int g_dla_flags;  // bit 5: a pipeline wait exceeded its limit

// Bounded wait. False when this or any other wait of the grid gave up. Its loop is a call: the
// kernels' dozens of waits inlined made them 100 KB long, and their warps wait for instructions as it is.
static __device__ __noinline__ bool wait_longer(uint32_t a, uint32_t parity) {
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (ptx::mbar_try(a, parity)) return true;
        if ((it & 63u) == 0) {
            if (*(volatile unsigned int *)&g_dla_flags != 0u) return false;
            if (clock64() - t0 > kWaitLimit) {
                atomicOr(&g_dla_flags, 32u);
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool wait_bar(uint32_t a, uint32_t parity) {
    return ptx::mbar_try(a, parity) || wait_longer(a, parity);
}
// for copies and products in flight after a failed wait: waits for them whatever the flag says
static __device__ __noinline__ void drain_bar(uint32_t a, uint32_t parity) {
    const long long t0 = clock64();
    while (!ptx::mbar_try(a, parity) && clock64() - t0 < kWaitLimit) {}
}
__device__ __forceinline__ void warp_arrive(uint32_t a) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(a);
}
inline cudaError_t read_flags(unsigned int *flags, bool reset, cudaStream_t stream) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(flags, g_dla_flags, sizeof(*flags), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbolAsync(g_dla_flags, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    return e;
}

// ---------------------------------------------------------------- segments
// Segment m of sequence n, of `seg` tokens, lives in slot cu[n] / seg + n + m: distinct over all
// segments and below n_tok / seg + n_seq, without a pass over the lengths on the host. Every sequence,
// an empty one too, has its first slot.
struct Segment {
    int seq, index;
    int64_t t0, len;   // len = 0 and index > 0: an unused slot
    bool last;         // the sequence ends in it
};
__device__ __forceinline__ int64_t segment_base(const int32_t *cu, int n, int seg) { return cu[n] / seg + n; }
__device__ __forceinline__ Segment find_segment(const int32_t *cu, int n_seq, int64_t slot, int seg) {
    int lo = 0, hi = n_seq - 1;  // largest n with segment_base(n) <= slot
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (segment_base(cu, mid, seg) <= slot) lo = mid; else hi = mid - 1;
    }
    const int64_t index = slot - segment_base(cu, lo, seg), t0 = cu[lo] + index * seg, left = cu[lo + 1] - t0;
    return {lo, (int)index, t0, left < 0 ? 0 : left < seg ? left : seg, left <= seg && (left > 0 || index == 0)};
}

// A state in the workspace, S^T by runs of four key channels: element (dk, dv) at
// (dk / 4) * 512 + dv * 4 + dk % 4, so that a thread with one dv writes 16 bytes beside its neighbour's
__host__ __device__ constexpr int state_floats(int dkp) { return dkp * 128; }

// ---------------------------------------------------------------- tiles
// The tensor maps of inputs [tokens, heads, d]: boxes of 64 tokens x 64 channels of one head.
struct TileMap {
    static PFN_cuTensorMapEncodeTiled_v12000 encoder() {
        static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
            void *ptr = nullptr;
            cudaDriverEntryPointQueryResult r;
            if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &r) != cudaSuccess ||
                r != cudaDriverEntryPointSuccess)
                ptr = nullptr;
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
        }();
        return fn;
    }
    // false: rows that a tensor copy cannot fetch (the kernels then load them by threads)
    static bool encode(CUtensorMap *m, const void *base, int64_t n_tok, int64_t stride, int heads, int d) {
        auto enc = encoder();
        if (!enc || n_tok == 0 || !gdr::rows_vec<__nv_bfloat16>(base, stride, d)) return false;
        const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)n_tok};
        const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
        const cuuint32_t box[3] = {64, 1, C}, step[3] = {1, 1, 1};
        return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
};

// One input of a kernel as its loader sees it
struct Source {
    const CUtensorMap *map;
    const __nv_bfloat16 *base;
    int64_t stride;
    int head, d, halves;   // halves of 64 channels in the tile; those past d stay as they are
    bool vec;              // 16-byte rows
};
// The tile of tokens t0 .. t0 + rows by one thread's tensor copies; a full tile only, so that no
// row of another sequence gets in
__device__ __forceinline__ void tile_by_copy(const Source &s, uint32_t dst, int64_t t0, uint32_t mbar) {
    for (int h = 0; h < s.halves; ++h) ptx::tma_load_3d(dst + h * kHalf, s.map, h * 64, s.head, (int)t0, mbar);
}
// the same by threads, rows past the end as zeros
static __device__ __noinline__ void tile_by_threads(const Source s, uint32_t dst, int64_t t0, int rows, int tid, int n) {
    const __nv_bfloat16 *p = s.base + t0 * s.stride + (int64_t)s.head * s.d;
    for (int h = 0; h < s.halves; ++h)
        gdr::load_tile<__nv_bfloat16, 128>(dst + h * kHalf, 0, p + h * 64, s.stride, rows, s.d - h * 64, s.vec, tid, n);
}

// The two loading warps' rows are in shared memory, for tensor-core operand reads too. Both warps come
// here for every such tile, whatever their waits said: the barrier counts on it.
__device__ __forceinline__ void tile_loaded(uint32_t mbar) {
    ptx::cp_async_commit();
    ptx::cp_async_wait0();
    ptx::fence_proxy_async();
    ptx::named_sync(1, 64);
    if ((threadIdx.x & 63) == 0) ptx::mbar_arrive(mbar);
}

// ---------------------------------------------------------------- gates
// Of one tile: running sums of g log2(e), the decays up to and with each token (gam), those past it
// times a factor as two bf16 planes, each twice in a word (del), the decay of all (whole)
struct TileGates {
    float2 G[C];
    float gam[C];
    uint2 del[C];
    float whole;
    float pad[3];
};
__device__ __forceinline__ uint2 planes_of(float x) {
    const uint32_t hi = ptx::pack_bf16(x, x), lo = ptx::pack_bf16(x - gdr::lo_f(hi), x - gdr::lo_f(hi));
    return make_uint2(hi, lo);
}
// Sums of g log2(e) in fixed point, 40 bits behind the point: exact, so that differences of
// neighbours stay exact after a long run of strong decays, and a scan's step is one addition (in two
// floats the six dependent additions of a two-sum made it the longest chain of a tile).
__device__ __forceinline__ int64_t fixed_exponent(float g) {
    const Two x = decay_exponent(g);
    return __float2ll_rn(x.hi * 1099511627776.f) + __float2ll_rn(x.lo * 1099511627776.f);
}
__device__ __forceinline__ float from_fixed(int64_t x) { return __ll2float_rn(x) * 9.094947017729282e-13f; }
// REV: del is the factor scale gam (the reverse walk's keys are scale gam q), else the decay past a token
template <bool REV>
__device__ __forceinline__ void form_gates(float2 g, float scale, TileGates *out) {
    const int lane = threadIdx.x & 31;
    const int64_t first = fixed_exponent(g.x), both = first + fixed_exponent(g.y);
    int64_t run = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
    }
    const int64_t total = __shfl_sync(0xffffffffu, run, 31);
    const int64_t G[2] = {run - both + first, run};
    float2 at[2];
    float gam[2];
    uint2 del[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float hi = from_fixed(G[i]);
        at[i] = make_float2(hi, from_fixed(G[i] - __float2ll_rn(hi * 1099511627776.f)));
        gam[i] = ex2(hi);
        del[i] = planes_of(REV ? scale * gam[i] : ex2(from_fixed(total - G[i])));
    }
    *reinterpret_cast<float4 *>(&out->G[2 * lane]) = make_float4(at[0].x, at[0].y, at[1].x, at[1].y);
    *reinterpret_cast<float2 *>(&out->gam[2 * lane]) = make_float2(gam[0], gam[1]);
    *reinterpret_cast<uint4 *>(&out->del[2 * lane]) = make_uint4(del[0].x, del[0].y, del[1].x, del[1].y);
    if (lane == 0) out->whole = ex2(from_fixed(total));
}
// Every tile's gates, by one warp. Their inputs go to `ring` (kAhead tiles of 64 floats) kAhead tiles
// ahead by asynchronous copies: a fetch takes longer than a tile's products. tile(n): the n-th tile of
// the walk; rows(c): its tokens; slot(n), ready(n) and done(n): where its gates go, the wait for that
// slot and the hand-over.
constexpr int kAhead = 8;
template <bool REV, typename Tile, typename Rows, typename Slot, typename Ready, typename Done>
__device__ __forceinline__ void walk_gates(const DlaArgs &p, float *ring, int64_t t0, int head, int nc, Tile tile, Rows rows,
                                           Slot slot, Ready ready, Done done) {
    const int r = 2 * (threadIdx.x & 31);
    auto fetch = [&](int n) {
        if (n < nc) {
            const int c = tile(n), len = rows(c);
            const float *g = p.g + (t0 + (int64_t)c * C + r) * p.g_stride + head;
            const uint32_t to = ptx::smem_u32(ring + n % kAhead * C + r);
            ptx::cp_async_4(to, r < len ? g : p.g, r < len ? 4 : 0);
            ptx::cp_async_4(to + 4, r + 1 < len ? g + p.g_stride : p.g, r + 1 < len ? 4 : 0);
        }
        ptx::cp_async_commit();
    };
#pragma unroll 1
    for (int n = 0; n < kAhead - 1; ++n) fetch(n);
#pragma unroll 1
    for (int n = 0; n < nc; ++n) {
        fetch(n + kAhead - 1);
        gdr::cp_async_wait<kAhead - 1>();
        const float2 g = *reinterpret_cast<const float2 *>(ring + n % kAhead * C + r);  // this lane's own copies
        ready(n);
        form_gates<REV>(g, p.scale, slot(n));
        done(n);
    }
}

// The planes of a tile's rows times their factors: hi = k d, lo the rest of the product and k times
// the factor's second plane. k d has 16 bits, so that its rest beside hi is exact. Eight channels a
// time, `dst` and `dst + plane`.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ void scale_rows(const char *src, char *dst, int plane, const TileGates &gate, int bytes,
                                           int tid, int n) {
#pragma unroll 4
    for (int i = tid; i < bytes / 16; i += n) {
        const uint4 k = reinterpret_cast<const uint4 *>(src)[i];
        const uint2 d = gate.del[(i >> 3) & (C - 1)];
        const uint32_t x[4] = {k.x, k.y, k.z, k.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = mul_bf16x2(x[e], d.x);
            lo[e] = fma_bf16x2(x[e], d.y, fma_bf16x2(x[e], d.x, hi[e] ^ 0x80008000u));
        }
        reinterpret_cast<uint4 *>(dst)[i] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        reinterpret_cast<uint4 *>(dst + plane)[i] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// two fp32 values as two packed planes
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = ptx::pack_bf16(x, y);
    lo = ptx::pack_bf16(x - gdr::lo_f(hi), y - gdr::hi_f(hi));
}

}  // namespace dla
}  // namespace kda
