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

// Bounded wait. False when this or any other wait of the grid gave up.
__device__ __forceinline__ bool wait_bar(uint32_t a, uint32_t parity) {
    if (ptx::mbar_try(a, parity)) return true;
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
__device__ __forceinline__ void tile_by_threads(const Source &s, uint32_t dst, int64_t t0, int rows, int tid, int n) {
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
// a tile's gates' inputs, two tokens a lane, ahead of their use
__device__ __forceinline__ void fetch_gates(const DlaArgs &p, int64_t t0, int len, int head, float *g) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 2 * (threadIdx.x & 31) + i;
        g[i] = r < len ? p.g[(t0 + r) * p.g_stride + head] : 0.f;
    }
}
// del: REV: factor gam (the reverse walk's keys are scale gamma q), else delta past the tile, and
// past `after` as well
template <bool REV>
__device__ __forceinline__ void form_gates(const float *g, float scale, TileGates *out) {
    const int lane = threadIdx.x & 31;
    Two s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) s[i] = decay_exponent(g[i]);
    s[1] = add(s[0], s[1]);
    const Two run = warp_scan(s[1]), total = last_lane(run);
    Two before = up(run, 1);
    if (lane == 0) before = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 2 * lane + i;
        const Two G = i ? run : add(before, s[0]);
        const float gam = exp2_of(G);
        out->G[r] = make_float2(G.hi, G.lo);
        out->gam[r] = gam;
        out->del[r] = planes_of(REV ? scale * gam : ex2((total.hi - G.hi) + (total.lo - G.lo)));
    }
    if (lane == 0) out->whole = exp2_of(total);
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
