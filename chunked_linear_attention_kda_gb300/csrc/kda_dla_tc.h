// Shared by the tensor-core kernels of linear attention with one decay per head (bf16 inputs):
// segments, tiles, gates and the walk over a segment that carries the state. Internal.
//
// A tile is 64 tokens of one head in column halves of 64 channels, each 64 rows of 128 bytes in the
// 128-byte swizzle of tensor copies, which tcgen05 reads K-major or MN-major as it stands. Operands
// that are not bf16 inputs are sums of bf16 planes: states and pair weights of two (within 2^-17 of the value),
// values times their decays as scale_values says.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_dla.h"

namespace kda {
namespace dla {

constexpr int C = 64;            // tokens of a tile
constexpr int kHalf = C * 128;   // bytes of a tile's 64 channels
constexpr uint32_t kWaitLimit = 3000000000u;  // SM cycles, about one and a half seconds

static __device__ unsigned int g_dla_flags;  // bit 5: a pipeline wait exceeded its limit

// Bounded wait. False when this or any other wait of the grid gave up.
__device__ __forceinline__ bool wait_bar(uint32_t a, uint32_t parity) {
    if (ptx::mbar_try(a, parity)) return true;
    const uint32_t t0 = clock();
#pragma unroll 1
    for (uint32_t it = 1;; ++it) {
        if (ptx::mbar_try(a, parity)) return true;
        if ((it & 63u) == 0) {
            if (*(volatile unsigned int *)&g_dla_flags != 0u) return false;
            if ((uint32_t)clock() - t0 > kWaitLimit) {
                atomicOr(&g_dla_flags, 32u);
                return false;
            }
        }
    }
}
// for copies and products in flight after a failed wait: waits for them whatever the flag says
__device__ __forceinline__ void drain_bar(uint32_t a, uint32_t parity) {
    const uint32_t t0 = clock();
    while (!ptx::mbar_try(a, parity) && (uint32_t)clock() - t0 < kWaitLimit) {}
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
__device__ __forceinline__ int64_t segment_base(const int32_t *cu, int n, int seg) {
    return (int64_t)((uint32_t)cu[n] / (uint32_t)seg) + n;
}
__device__ __forceinline__ Segment find_segment(const int32_t *cu, int n_seq, int64_t slot, int seg) {
    int lo = 0, hi = n_seq - 1;  // largest n with segment_base(n) <= slot
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (segment_base(cu, mid, seg) <= slot) lo = mid; else hi = mid - 1;
    }
    const int64_t index = slot - segment_base(cu, lo, seg), t0 = cu[lo] + index * seg, left = cu[lo + 1] - t0;
    return {lo, (int)index, t0, left < 0 ? 0 : left < seg ? left : seg, left <= seg && (left > 0 || index == 0)};
}

// The j-th longest segment of a call, by a whole block: CTAs begin in the order of their numbers, and short
// segments after the long ones fill the SMs evenly (20K tokens in 12 sequences, 32 heads: 195 us in
// the sequences' order, 165 so). `scratch`: shared memory that nothing else uses before the block's next barrier.
// One sequence's segments are of one length; beyond 256 the order of so many units matters little.
struct Ordered { Segment sg; int64_t slot; };
__device__ __forceinline__ Ordered jth_longest(const int32_t *cu, int n_seq, int64_t j, int64_t slots, int seg, char *scratch) {
    if (n_seq == 1 || slots > 256) return {find_segment(cu, n_seq, j, seg), j};
    Ordered *out = reinterpret_cast<Ordered *>(scratch);
    int *len = reinterpret_cast<int *>(scratch + sizeof(Ordered));
    const int t = threadIdx.x, n = (int)slots;
    Segment mine{};
    if (t < n) {
        mine = find_segment(cu, n_seq, t, seg);
        len[t] = (int)mine.len;
    }
    __syncthreads();
    if (t < n) {
        int rank = 0;
        for (int i = 0; i < n; ++i) rank += len[i] > (int)mine.len || (len[i] == (int)mine.len && i < t);
        if (rank == (int)j) *out = {mine, t};
    }
    __syncthreads();
    const Ordered got = *out;
    ptx::fence_proxy_async();  // tensor copies come next
    __syncthreads();
    return got;
}

// A state in the workspace, S^T by runs of four key channels: element (dk, dv) at
// (dk / 4) * 512 + dv * 4 + dk % 4, so that a thread with one dv writes 16 bytes beside its neighbour's
__host__ __device__ constexpr int state_floats(int dkp) { return dkp * 128; }

// ---------------------------------------------------------------- tiles
// The tensor maps of inputs [tokens, heads, d]: boxes of `rows` tokens x 64 channels of one head.
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
    static bool encode(CUtensorMap *m, const void *base, int64_t n_tok, int64_t stride, int heads, int d, int rows = C) {
        auto enc = encoder();
        if (!enc || n_tok == 0 || !gdr::rows_vec<__nv_bfloat16>(base, stride, d)) return false;
        const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)n_tok};
        const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
        const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows}, step[3] = {1, 1, 1};
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
// The tile of the tokens from t0 on by one thread's tensor copies
__device__ __forceinline__ void tile_by_copy(const Source &s, uint32_t dst, int64_t t0, uint32_t mbar) {
    for (int h = 0; h < s.halves; ++h) ptx::tma_load_3d(dst + h * kHalf, s.map, h * 64, s.head, (int)t0, mbar);
}
// Its rows from `rows` on as zeros, by a warp: they are another sequence's. `pitch`: bytes of a half.
__device__ __forceinline__ void clear_rows(uint32_t dst, int halves, int pitch, int rows, int total) {
    const uint32_t zero[4] = {0, 0, 0, 0};
    for (int h = 0; h < halves; ++h)
        for (int i = rows * 8 + (threadIdx.x & 31); i < total * 8; i += 32) gdr::st_shared_16(dst + h * pitch + i * 16, zero);
}
// the same of `n` inputs by threads, rows past the end as zeros
__device__ __forceinline__ void tiles_by_threads(const Source *inputs, const uint32_t *dst, int n, int64_t t0, int rows,
                                                 int tid, int threads) {
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const Source &s = inputs[i];
        const __nv_bfloat16 *p = s.base + t0 * s.stride + (int64_t)s.head * s.d;
#pragma unroll 1
        for (int h = 0; h < s.halves; ++h)
            gdr::load_tile<__nv_bfloat16, 128>(dst[i] + h * kHalf, 0, p + h * 64, s.stride, rows, s.d - h * 64, s.vec, tid, threads);
    }
}
// a loading warp's rows are in shared memory, for tensor-core operand reads too
__device__ __forceinline__ void rows_loaded() {
    ptx::cp_async_commit();
    ptx::cp_async_wait0();
    ptx::fence_proxy_async();
    __syncwarp();
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t mbar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(mbar) : "memory");
}

// ---------------------------------------------------------------- gates
// Of one tile and head, formed for all tiles by a launch of their own (kda_dla_fwd.cu) and copied in with the
// tile: running sums of g log2(e), whole number and rest, scale times the decays up to and with each token (gam), the decays
// past each (del), the decay of all in two parts (whole) and its exponent in fixed point (sum). Formed beside the products by one warp they
// were the longest chain of a tile (1700 cycles of scans and conversions).
struct TileGates {
    float2 G[C];
    float gam[C], del[C];
    Two whole;
    int64_t sum;
};
static_assert(sizeof(TileGates) % 16 == 0, "copied in bulk");
// The gates of tile c of a sequence lie at slot_base(cu, sequence) + c, as in kda_gdr.h
__device__ __forceinline__ const TileGates *gates_of(const TileGates *all, const DlaArgs &p, int seq, int64_t c, int head) {
    return all + ((slot_base(p.cu_seqlens, seq) + c) * p.n_heads + head);
}
// Sums of g log2(e) in fixed point, 44 bits behind the point: exact, so that differences of neighbours
// stay exact after a long run of strong decays, and a scan's step is one addition. An exponent is cut off
// after 20 bits, towards zero: what is left is exact and of its sign, however small the exponent is, and
// gives the other 24. (Rounded down, the rest of a small negative one is near 1 and loses its last places, the
// same at every token of a constant rate: a state of 64K tokens at -3.7e-5 was off by 9e-5 of its norm.) By
// conversions of 32 bits alone: those of 64 are as slow as fp64 on this part (gates of 64K tokens of 32
// heads: 31 us with them).
constexpr int kPoint = 44;
__device__ __forceinline__ int64_t fixed_exponent(float g) {
    const Two x = decay_exponent(g);
    const float y = x.hi * 0x1p20f, n = truncf(y);
    return ((int64_t)(int)n << 24) + __float2int_rn(fmaf(x.lo, 0x1p20f, y - n) * 0x1p24f);
}
// the nearest whole number and the rest, to 2^-26 and to 2^-37 near 0
__device__ __forceinline__ float2 from_fixed(int64_t x) {
    const int n = (int)((x + ((int64_t)1 << (kPoint - 1))) >> kPoint);
    const int64_t f = x - ((int64_t)n << kPoint);
    return make_float2((float)n, fmaf((float)(int)(f >> 32), 0x1p-12f, (float)(uint32_t)f * 0x1p-44f));
}
__device__ __forceinline__ float exp2_fixed(int64_t x) {
    const float2 y = from_fixed(x);
    return ex2(y.x) * ex2(y.y);
}
__device__ __forceinline__ Two exp2_fixed_parts(int64_t x) {
    const float2 y = from_fixed(x);
    return exp2_parts(y.x, y.y);
}
// NaN where a tile's gates are, which its sum cannot show
__device__ __forceinline__ float nan_of(const TileGates &g) { return g.whole.hi - g.whole.hi; }
// A tile's gates by one warp, two tokens a lane; tokens past the end have g = 0. A g that is NaN, or past what
// the sums hold (whose decay is infinite), makes all of them NaN: as a fixed point number it would pass for a 0.
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
    const int64_t before = run - both + first;
    const float bad = __any_sync(0xffffffffu, !(g.x <= 1e3f && g.y <= 1e3f)) ? __int_as_float(0x7fffffff) : 0.f;
    float2 a = from_fixed(before), b = from_fixed(run);
    a.x += bad;
    b.x += bad;
    reinterpret_cast<float4 *>(out->G)[lane] = make_float4(a.x, a.y, b.x, b.y);
    reinterpret_cast<float2 *>(out->gam)[lane] = make_float2(scale * ex2(a.x) * ex2(a.y), scale * ex2(b.x) * ex2(b.y));
    reinterpret_cast<float2 *>(out->del)[lane] = make_float2(exp2_fixed(total - before) + bad, exp2_fixed(total - run) + bad);
    if (lane == 0) {
        const Two whole = exp2_fixed_parts(total);
        out->whole = {whole.hi + bad, whole.lo};
        out->sum = total;
    }
}

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
// A tile's values times their tokens' factors, V'^T, as NP planes in tensor memory (columns `to` + 32 i .. + 31,
// two tokens a column). Two, by bf16 arithmetic: v times the factor's first plane has 16 bits, so that its rest
// beside the first plane is exact, and the second takes that and v times the factor's second plane: within
// 2^-14.8 of the product (4 instructions a pair of values; by fp32 arithmetic, 10, they are within 2^-17, and 64K
// tokens of 32 heads take 665 us instead of 625). Three, by fp32 arithmetic: every plane is what is left of
// the product, which one FMA forms exactly, rounded to bf16: within 2^-25. (In bf16 arithmetic what is left after two is
// not always exact, and three were within 2^-16.) By one warp of each quarter of the lanes, 32 value channels. As an
// A operand there it costs shared memory, which bounds these kernels, one read of the tile; as planes in
// shared memory for either operand a read, a write a plane and a read each. `ready` waits until the planes may be
// written; the first are formed before it.
template <int NP, typename Ready>
__device__ __forceinline__ void scale_values(uint32_t tile, uint32_t tmem, uint32_t to, const float *factor, float more, Ready ready) {
    const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3;
    const uint32_t col = (lane >> 3 & 1) * 8;  // matrices 0, 1: channels 0..7 and 8..15 of eight tokens; 2, 3: of the next eight
    constexpr uint32_t minus = 0x80008000u;
#pragma unroll 1
    for (int t0 = 0; t0 < C; t0 += 32) {
        float2 f[4];  // of the tokens t0 + 8 n + 2 (lane % 4) and the next
        uint32_t f0[4], f1[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            f[n] = *reinterpret_cast<const float2 *>(factor + t0 + 8 * n + 2 * (lane & 3));
            f[n].x *= more;
            f[n].y *= more;
            if constexpr (NP == 2) {
                f0[n] = ptx::pack_bf16(f[n].x, f[n].y);
                f1[n] = ptx::pack_bf16(f[n].x - gdr::lo_f(f0[n]), f[n].y - gdr::hi_f(f0[n]));
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int dv = 32 * q + 16 * h + col;
            uint32_t x[NP][8];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int tok = t0 + 16 * n + (lane >> 4) * 8 + (lane & 7);
                ptx::ldsm_x4_t(tile + gdr::key_off(tok, dv), x[0][4 * n], x[0][4 * n + 1], x[0][4 * n + 2], x[0][4 * n + 3]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t v = x[0][i];
                if constexpr (NP == 2) {
                    x[0][i] = mul_bf16x2(v, f0[i >> 1]);
                    x[1][i] = fma_bf16x2(v, f1[i >> 1], fma_bf16x2(v, f0[i >> 1], x[0][i] ^ minus));
                } else {
                    const float a = gdr::lo_f(v), b = gdr::hi_f(v);
                    const float2 y = f[i >> 1];
                    x[0][i] = ptx::pack_bf16(a * y.x, b * y.y);
                    const float ra = fmaf(a, y.x, -gdr::lo_f(x[0][i])), rb = fmaf(b, y.y, -gdr::hi_f(x[0][i]));
                    x[1][i] = ptx::pack_bf16(ra, rb);
                    x[2][i] = ptx::pack_bf16(ra - gdr::lo_f(x[1][i]), rb - gdr::hi_f(x[1][i]));
                }
            }
            if (t0 == 0 && h == 0) ready();
            const uint32_t at = tmem + ((uint32_t)(32 * q + 16 * h) << 16) + to + t0 / 2;
#pragma unroll
            for (int i = 0; i < NP; ++i) ptx::tmem_st_half4(at + 32 * i, x[i]);
        }
    }
    ptx::tmem_st_wait();
}

// two fp32 values as two packed planes
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = ptx::pack_bf16(x, y);
    lo = ptx::pack_bf16(x - gdr::lo_f(hi), y - gdr::hi_f(hi));
}

}  // namespace dla
}  // namespace kda
