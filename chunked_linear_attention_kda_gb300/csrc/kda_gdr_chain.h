// The serial chains over a sequence's chunks: the forward's (with its output, or for the
// backward pass with a record of every chunk's state) and the backward's reverse one. The
// mathematics is in kda_gdr_fwd.cu and kda_gdr_bwd.cu. Internal; not part of the C ABI.
//
// A CTA of nine warps advances 16 value channels per pair of state warps through a sequence:
//   state warps   S^T (16 x d_k) is held as bf16 planes by both warps of a pair and in fp32 by
//                 halves of d_k. An accumulator tile of mma.sync lies in registers as the A
//                 operand of the next product, so a warp goes S^T -> Y^T -> Z^T -> U^T without
//                 leaving its registers; each warp of a pair takes one half of the chunk's
//                 tokens, then one half of d_k in the update of S, and the pair exchanges its
//                 halves of Z^T, U^T and S^T through shared memory at barriers of 64 threads.
//   the last warp one thread loads: tensor copies of whole chunks, bulk copies of the chunk
//                 terms and of tile images, into rings of stages.
// With two pairs the other four warps take what the serial path need not wait for: the output
// O (from copies of S^T and U^T left in shared memory) or, in reverse, dO^T P and (gamma dO)^T
// Q, handed to the state warps ahead of their use. With four pairs (the backward pass, when
// there are more chains than SMs) the state warps do that themselves: a step is longer but
// covers twice the channels, and each scheduler has two state warps to choose from.
// Per chunk the state warps of a pair issue 146 and 170 mma.sync m16n8k16 (bf16, d_k = 128, forward)
// of 8 cycles each on their schedulers' tensor pipes, and the helper beside each another 94: 2100
// cycles bound a step from below. It takes 3700 (64K tokens, 32 heads: 1024 steps in 1.98 ms); the rest
// is the latency of dependent products (20 cycles each) and of four hand-overs. Measured and dropped,
// against 1.83 ms with S0 and P in one plane in the output: loops over the state's tiles that are not
// unrolled (3.0 ms), Y begun with the pair's own half before the barrier (1.92 ms).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_gdr.h"

namespace kda {
namespace gdr {

enum class Mode { kForward, kStates, kReverse };
constexpr int kChainThreads = 288;
constexpr long long kWaitLimit = 4000000000LL;  // SM cycles, about two seconds

static __device__ unsigned int g_gdr_flags;  // bit 4: a pipeline wait exceeded its limit

// Bounded wait. False when this or any other wait of the grid gave up.
__device__ __forceinline__ bool wait_bar(uint32_t a, uint32_t parity) {
    if (ptx::mbar_try(a, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (ptx::mbar_try(a, parity)) return true;
        if ((it & 63u) == 0) {
            if (*(volatile unsigned int *)&g_gdr_flags != 0u) return false;
            if (clock64() - t0 > kWaitLimit) {
                atomicOr(&g_gdr_flags, 16u);
                return false;
            }
        }
    }
}
// for copies in flight after a failed wait: waits for them whatever the flag says, as long again
static __device__ __noinline__ void drain_bar(uint32_t a, uint32_t parity) {
    const long long t0 = clock64();
    while (!ptx::mbar_try(a, parity) && clock64() - t0 < kWaitLimit) {}
}
// whether the phase is complete, without waiting
__device__ __forceinline__ bool test_bar(uint32_t a, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(a), "r"(parity) : "memory");
    return ok != 0;
}
// every lane of a warp waits; all leave with the same answer
__device__ __forceinline__ bool warp_wait(uint32_t a, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_bar(a, parity));
}
__device__ __forceinline__ void warp_arrive(uint32_t a) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(a);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t mbar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(mbar) : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
                 : "memory");
}
// one 16 x 16 block of an A-operand fragment to a swizzled tile, `a` the address of lane's row
__device__ __forceinline__ void store_block(uint32_t a, const uint32_t *f) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(f[0]), "r"(f[1]),
                 "r"(f[2]), "r"(f[3]) : "memory");
}
__device__ __forceinline__ void bulk_wait0() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Shared memory (offsets from a 1024-byte boundary). Ring 1 (state warps): K, X, gates and,
// forward, V. Ring 2 (the others): Q, P, gates and, reverse, dO. Per pair: Sx the planes of
// S^T and Uo U^T itself (both read by the output warps), Ux the scaled planes of U^T that
// the pair exchanges, Zx those of the first half's Z^T; Hand the accumulators handed over in
// reverse; Keep the staging of the records that go to the workspace (bf16; fp32 inputs, whose
// tiles leave no room for it, store them from registers).
template <int NI, int DKP, int NS, Mode M, int PAIRS>
struct ChainSmem {
    static constexpr bool kHelp = PAIRS == 2;
    static constexpr bool kOut = M == Mode::kForward, kRev = M == Mode::kReverse;
    static constexpr int kKey = NI * C * DKP * 2, kSlice = NI * C * 64, kVal = PAIRS / 2 * kSlice;
    static constexpr int kX = NS * kTri, kP = NS * kTri;
    static constexpr int kGate = kChainGates * 4;
    // ring 1
    static constexpr int K = 0, V = K + kKey, X = V + (kRev ? 0 : kVal), Gate1 = X + kX;
    static constexpr int kStage1 = (Gate1 + kGate + 1023) / 1024 * 1024;
    // As many stages as fit (three planes, 512 tokens of 4 heads, backward: 77 us with two, 85 with
    // one); for fp32 with d_k above 64 that is one, and a step waits for its chunk's copy.
    static constexpr int N1 = NS == 2 ? (kRev ? 2 : 3) : NI == 1 || DKP == 64 ? 2 : 1;
    // ring 2
    static constexpr int Q = 0, dO = Q + kKey, P = dO + (kRev ? kVal : 0), Gate2 = P + kP;
    static constexpr int kStage2 = (Gate2 + kGate + 1023) / 1024 * 1024;
    static constexpr int N2 = M == Mode::kStates ? 0 : NS == 2 && kHelp ? 2 : 1;
    // per pair
    static constexpr int NH = kOut ? 2 : 1;            // buffers of Sx and Uo
    static constexpr int kSx = NS * (DKP / 16) * 512, kUx = NS * 4 * 512, kZx = NS * 2 * 512;
    static constexpr int kUo = kOut ? C * 64 : 0;
    static constexpr int kHandG = DKP * 64, kHand = kRev && kHelp ? kHandG + C * 64 : 0;
    static constexpr int kKeepP = 16 * (DKP + C) * 2, kKeepV = 16 * DKP * 2;  // a plane; U or E in it
    static constexpr int kKeep = kOut || NI == 3 ? 0 : scan_part(NS, DKP);
    static constexpr int Sx = 0, Uo = Sx + NH * kSx, Ux = Uo + NH * kUo, Zx = Ux + kUx, Hand = Zx + kZx, Keep = Hand + kHand;
    static constexpr int kPair = Keep + kKeep;
    static constexpr int Ring2 = N1 * kStage1, Pairs = Ring2 + N2 * kStage2, Bars = Pairs + PAIRS * kPair;
    static constexpr int kBars = 2 * N1 + 2 * N2 + (kHelp ? 4 * NH : 0);
    static constexpr int kBytes = Bars + 8 * kBars + 1024;        // the base is rounded up to 1024
    static_assert(kBytes <= 226 * 1024, "fits an SM");
    static_assert(kKey % 1024 == 0 && kSlice % 1024 == 0, "tensor copies land on swizzle boundaries");
};

// The tensor maps of q, k and v (and dout); make() is false when the inputs need images.
struct ChainMaps {
    CUtensorMap q, k, v, dout;
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
    // boxes of 64 tokens x `width` channels of one head
    static bool encode(CUtensorMap *m, const void *base, int64_t n_tok, int64_t stride, int heads, int d, int width) {
        auto enc = encoder();
        if (!enc) return false;
        const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)n_tok};
        const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
        const cuuint32_t box[3] = {(cuuint32_t)width, 1, C}, step[3] = {1, 1, 1};
        return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, width == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
    template <typename T>
    bool make(const GdrArgs &p, bool with_dout) {
        if (sizeof(T) != 2 || p.n_tok == 0) return false;
        if (!rows_vec<T>(p.q, p.q_stride, p.d_k) || !rows_vec<T>(p.k, p.k_stride, p.d_k) ||
            !rows_vec<T>(p.v, p.v_stride, p.d_v))
            return false;
        const int64_t vs = (int64_t)p.n_heads * p.d_v;
        if (with_dout && !rows_vec<T>(p.dout, vs, p.d_v)) return false;
        return encode(&q, p.q, p.n_tok, p.q_stride, p.n_k_heads, p.d_k, 64) &&
               encode(&k, p.k, p.n_tok, p.k_stride, p.n_k_heads, p.d_k, 64) &&
               encode(&v, p.v, p.n_tok, p.v_stride, p.n_heads, p.d_v, 32) &&
               (!with_dout || encode(&dout, p.dout, p.n_tok, vs, p.n_heads, p.d_v, 32));
    }
};

inline unsigned chain_blocks(const GdrArgs &p, int pairs) {
    return (unsigned)((p.d_v + 16 * pairs - 1) / (16 * pairs)) * p.n_heads * p.n_seq;
}
// Pairs of the backward pass's chains (d_k = d_v = 128). Two pairs end a step sooner (3500 cycles
// forward, 4600 in reverse, against 4450 and 7800), four cover twice the channels: worth it
// once the CTAs of two pairs are more than one and a half waves. With 128 CTAs of two pairs
// (4K tokens, 16 heads) the backward pass takes 272 us with two and 371 with four, with 192
// (24 heads) 403 and 415, with 256 (2K tokens, 32 heads) 249 and 248, with 512 (two sequences of
// 8K tokens, 32 heads) 1710 and 1501. The forward pass gains nothing from four: the output would
// lengthen its step to over 6500 cycles.
inline int scan_pairs(const GdrArgs &p) {
    constexpr unsigned kSMs = 152;
    return p.d_v > 32 && 2 * chain_blocks(p, 2) > kSMs + kSMs / 2 ? 4 : 2;
}

// The sequence of the given rank, longest first (ties by index): the longest chains start first, so
// that none is left alone at the end. Every CTA finds its own, which costs it n_seq^2 comparisons: up to
// 64 sequences; more are taken in order, and with more CTAs the end weighs less. 64K tokens of 32 heads
// in sequences of lengths that differ by up to 150, the longest last, forward: 16 of them 2140 us ranked and
// 2328 in order, 64 of them 2341 and 2350, 128 of them 2683 and 2523, 512 of them 11026 and 3857.
constexpr int kRanked = 64;
__device__ __forceinline__ int ranked_sequence(const int32_t *cu, int n_seq, int rank, int *shared) {
    if (n_seq == 1 || n_seq > kRanked) return rank;
    // one pass at most; as a branch it costs the chains registers (8K x 2 backward: 1525 us, 1505 so)
    for (int s = threadIdx.x; s < n_seq; s += blockDim.x) {
        const int len = cu[s + 1] - cu[s];
        int r = 0;
        for (int o = 0; o < n_seq; ++o) {
            const int l = cu[o + 1] - cu[o];
            r += l > len || (l == len && o < s);
        }
        if (r == rank) *shared = s;
    }
    __syncthreads();
    return *shared;
}

// ---- products of the state warps

// y (16 x 16, tokens n0 ..) = S^T K^T from the planes of S^T, those of half h of the key channels
// first; with two planes the lower one's products run on accumulators of their own, so that no
// product waits for the one before it
template <int NI, int NS, int DKP>
__device__ __forceinline__ void state_times_keys(const uint32_t (*a)[DKP / 16][4], uint32_t k, int h, int n0, float (*y)[4]) {
    float lo[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[0][i] = y[1][i] = lo[0][i] = lo[1][i] = 0.f;
#pragma unroll
    for (int kx = 0; kx < DKP / 16; ++kx) {
        const int half = kx < DKP / 32 ? h : 1 - h;
        uint32_t b[NI][4];
#pragma unroll
        for (int q = 0; q < NI; ++q) key_b(k + q * C * DKP * 2, n0, half * (DKP / 2) + (kx % (DKP / 32)) * 16, b[q]);
        if constexpr (NS == 3) {
            uint32_t x[NS][4];
#pragma unroll
            for (int q = 0; q < NS; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[q][i] = a[q][kx][i];
            product<NS, NI, 3>(y, x, b);
        } else {
            ptx::mma16816(y[0], a[0][kx], b[0][0], b[0][1]);
            ptx::mma16816(y[1], a[0][kx], b[0][2], b[0][3]);
            ptx::mma16816(lo[0], a[1][kx], b[0][0], b[0][1]);
            ptx::mma16816(lo[1], a[1][kx], b[0][2], b[0][3]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[0][i] += lo[0][i];
        y[1][i] += lo[1][i];
    }
}
// S (16 x DKP / 2, key channels c0 ..) += u^T K over tokens k0 .. k0 + 15, u^T as planes
template <int NI, int NS, int DKP>
__device__ __forceinline__ void add_values_keys(const uint32_t (*a)[4], uint32_t k, int k0, int c0, float (*S)[4]) {
#pragma unroll
    for (int n = 0; n < DKP / 32; ++n) {
        uint32_t b[NI][4];
#pragma unroll
        for (int q = 0; q < NI; ++q) key_b_t(k + q * C * DKP * 2, k0, c0 + n * 16, b[q]);
        product<NS, NI, NS>(&S[2 * n], a, b);
    }
}
// u (16 x 16, block n of the result's tokens) += a X over block k of the contraction
template <int NS, bool REV>
__device__ __forceinline__ void add_times_x(const uint32_t (*a)[4], uint32_t x, int k, int n, float (*u)[4]) {
    uint32_t b[NS][4];
#pragma unroll
    for (int q = 0; q < NS; ++q) {
        if (REV) frag_b_t<32>(x + q * kTri + tri_block(k, n), 0, 0, b[q]);
        else frag_b<32>(x + q * kTri + tri_block(n, k), 0, 0, b[q]);
    }
    product<NS, NS, NS>(u, a, b);
}
// planes of a 16 x 16 block to and from shared memory, 16 bytes a lane, planes `plane` apart
template <int NS>
__device__ __forceinline__ void put_block(char *p, int plane, const uint32_t (*a)[4]) {
#pragma unroll
    for (int q = 0; q < NS; ++q)
        *reinterpret_cast<uint4 *>(p + q * plane + (threadIdx.x & 31) * 16) = make_uint4(a[q][0], a[q][1], a[q][2], a[q][3]);
}
template <int NS>
__device__ __forceinline__ void get_block(const char *p, int plane, uint32_t (*a)[4]) {
#pragma unroll
    for (int q = 0; q < NS; ++q) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p + q * plane + (threadIdx.x & 31) * 16);
        a[q][0] = x.x; a[q][1] = x.y; a[q][2] = x.z; a[q][3] = x.w;
    }
}
// ---- the output, 32 tokens x 16 value channels: o[m][n], token blocks h and 3 - h, whose products
// with the lower triangle P are five blocks for either h
__device__ __forceinline__ int out_block(int h, int m) { return m ? 3 - h : h; }

// the A-operand planes of a 16 x 16 block as the B operand of the transposed product
template <int NP>
__device__ __forceinline__ void as_b(const uint32_t (*a)[4], uint32_t (*b)[4]) {
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        b[q][0] = a[q][0]; b[q][1] = a[q][2]; b[q][2] = a[q][1]; b[q][3] = a[q][3];
    }
}
// o += Q S0, key channels of block kx; a the planes of S^T
template <int NI, int NS, int DKP>
__device__ __forceinline__ void add_queries(const uint32_t (*a)[4], uint32_t q, int h, int kx, float (*o)[2][4]) {
    uint32_t b[NS][4];
    as_b<NS>(a, b);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        uint32_t f[NI][4];
#pragma unroll
        for (int x = 0; x < NI; ++x) key_a(q + x * C * DKP * 2, out_block(h, m) * 16, kx * 16, f[x]);
        product<NI, NS, NS>(o[m], f, b);
    }
}
__device__ __forceinline__ void scale_output(float (*o)[2][4], const float *gate, float scale, int h) {
    const int gr = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int r = out_block(h, m) * 16 + gr;
        const float g0 = scale * gate[r], g1 = scale * gate[r + 8];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            o[m][n][0] *= g0; o[m][n][1] *= g0; o[m][n][2] *= g1; o[m][n][3] *= g1;
        }
    }
}
// o += P U; uo the pair's U^T (fp32 accumulators)
template <int NS>
__device__ __forceinline__ void add_p_values(const char *uo, uint32_t pt, int h, float (*o)[2][4]) {
#pragma unroll
    for (int kx = 0; kx < 4; ++kx) {
        if (kx > 3 - h) break;
        uint32_t a[NS][4];
        float u[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float4 x = *reinterpret_cast<const float4 *>(uo + ((2 * kx + n) * 32 + (threadIdx.x & 31)) * 16);
            u[n][0] = x.x; u[n][1] = x.y; u[n][2] = x.z; u[n][3] = x.w;
        }
        acc_to_a<NS>(u, a);
        uint32_t b[NS][4];
        as_b<NS>(a, b);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (kx > out_block(h, m)) continue;
            uint32_t f[NS][4];
#pragma unroll
            for (int q = 0; q < NS; ++q) frag_a<32>(pt + q * kTri + tri_block(out_block(h, m), kx), 0, 0, f[q]);
            product<NS, NS, NS>(o[m], f, b);
        }
    }
}
template <typename T>
__device__ __forceinline__ void store_output(T *out, const float (*o)[2][4], int row0, int h, int v0, int64_t tok0,
                                             int len, int head, const GdrArgs &p, bool wide) {
    const int gr = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = row0 + out_block(h, m) * 16 + gr + x * 8;
            if (r >= len) continue;
            T *row = out + ((tok0 + r) * p.n_heads + head) * p.d_v;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int v = v0 + n * 8 + tq * 2;
                if (v < p.d_v) put2(row + v, o[m][n][x * 2], o[m][n][x * 2 + 1], wide, v + 1 < p.d_v);
            }
        }
}

// ---- the reverse chain's products with dO (a slice of 32 channels; channel half w of it)

template <int NI>
__device__ __forceinline__ void frag_dout(uint32_t dout, int kx, int w, uint32_t (*a)[4]) {
#pragma unroll
    for (int q = 0; q < NI; ++q) frag_a_t<64>(dout + q * C * 64, kx * 16, w * 16, a[q]);
}
// y (16 x 16) += dO^T P, P's block at `pt`
template <int NI, int NS>
__device__ __forceinline__ void add_dout_p(const uint32_t (*a)[4], uint32_t pt, float (*y)[4]) {
    uint32_t b[NS][4];
#pragma unroll
    for (int q = 0; q < NS; ++q) frag_b_t<32>(pt + q * kTri, 0, 0, b[q]);
    product<NI, NS, NS>(y, a, b);
}
// planes of (s gamma dO)^T
template <int NI, int NS>
__device__ __forceinline__ void scale_dout(const uint32_t (*a)[4], const float *gate, float scale, int kx, uint32_t (*d)[4]) {
    const int tq = threadIdx.x & 3;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 ga = *reinterpret_cast<const float2 *>(gate + kx * 16 + (j >> 1) * 8 + tq * 2);
        float x = 0.f, z = 0.f;
#pragma unroll
        for (int q = 0; q < NI; ++q) {
            x += lo_f(a[q][j]);
            z += hi_f(a[q][j]);
        }
        uint32_t sp[NS];
        split2<NS>(x * (scale * ga.x), z * (scale * ga.y), sp);
#pragma unroll
        for (int q = 0; q < NS; ++q) d[q][j] = sp[q];
    }
}

template <int N>
__device__ __forceinline__ void zero(float (*x)[4]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = 0.f;
}
template <int NT>
__device__ __forceinline__ void load_state(float (*S)[4], const float *src, int c0, int v0, int d_k, int d_v) {
    const int gr = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + n * 8 + tq * 2 + (i & 1), v = v0 + gr + (i >> 1) * 8;
            S[n][i] = src && c < d_k && v < d_v ? src[(size_t)c * d_v + v] : 0.f;
        }
}
template <int NT>
__device__ __forceinline__ void store_state(const float (*S)[4], float *dst, int c0, int v0, int d_k, int d_v) {
    const int gr = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + n * 8 + tq * 2 + (i & 1), v = v0 + gr + (i >> 1) * 8;
            if (c < d_k && v < d_v) dst[(size_t)c * d_v + v] = S[n][i];
        }
}

// One CTA's chain; `block` counts channel blocks, then heads, then sequences (longest first).
// tm_v is dout's map in reverse; `values` and `im` as given to the chunk terms.
template <typename T, int DKP, int NS, Mode M, int PAIRS>
__device__ __forceinline__ void chain(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                      const GdrArgs &p, const Images &im, int values, int block, float scale,
                                      bool wide_out) {
    constexpr int NI = InputPlanes<T>::N;
    using L = ChainSmem<NI, DKP, NS, M, PAIRS>;
    constexpr int NT = DKP / 16, KX = DKP / 16, N1 = L::N1, N2 = L::N2, NH = L::NH;
    constexpr bool kOut = L::kOut, kRev = L::kRev, kHelp = L::kHelp;
    extern __shared__ __align__(1024) char smem_raw[];
    char *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    __shared__ int ranked;
    wait_for_previous_kernel();  // the chunk terms
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tq = lane & 3;
    const int n_blk = (p.d_v + 16 * PAIRS - 1) / (16 * PAIRS);
    const int blk = block % n_blk, sh = block / n_blk;
    const int head = sh % p.n_heads, kh = head / (p.n_heads / p.n_k_heads);
    const int seq = ranked_sequence(p.cu_seqlens, p.n_seq, sh / p.n_heads, &ranked);
    const int64_t tok0 = p.cu_seqlens[seq];
    const int len = (int)(p.cu_seqlens[seq + 1] - tok0);
    const int n_chunks = (len + C - 1) / C;
    const int64_t slot0 = slot_base(p.cu_seqlens, seq);
    // pair w of the CTA's 16-channel halves; half h of its tokens and of d_k
    const int w = (warp >> 1) & (PAIRS - 1), h = warp & 1, v0 = (blk * PAIRS + w) * 16;
    const size_t st_at = ((size_t)seq * p.n_heads + head) * p.d_k * p.d_v;
    char *ws = static_cast<char *>(p.workspace);
    char *pair = smem + L::Pairs + w * L::kPair;

    auto bar = [&](int i) { return base + L::Bars + 8 * i; };
    auto full1 = [&](int s) { return bar(s); };
    auto empty1 = [&](int s) { return bar(N1 + s); };
    auto full2 = [&](int s) { return bar(2 * N1 + s); };
    auto empty2 = [&](int s) { return bar(2 * N1 + N2 + s); };
    auto hfull = [&](int b) { return bar(2 * N1 + 2 * N2 + b * 2 + w); };
    auto hempty = [&](int b) { return bar(2 * N1 + 2 * N2 + 2 * NH + b * 2 + w); };
    if (tid == 0) {
        for (int s = 0; s < N1; ++s) { ptx::mbar_init(full1(s), 1); ptx::mbar_init(empty1(s), 2 * PAIRS); }
        for (int s = 0; s < N2; ++s) { ptx::mbar_init(full2(s), 1); ptx::mbar_init(empty2(s), kHelp ? 4 : 8); }
        if (kHelp)
            for (int b = 0; b < 4 * NH; ++b) ptx::mbar_init(bar(2 * N1 + 2 * N2 + b), 2);
        ptx::mbar_init_fence();
    }
    __syncthreads();
    // step i works on chunk at(i)
    auto at = [&](int i) { return kRev ? n_chunks - 1 - i : i; };

    if (warp == 8) {
        // ------------------------------------------------ loads
        if (lane == 0) {
            const size_t rec = Images::record(NI, DKP, p.d_v, p.n_k_heads, p.n_heads, values);
            const size_t kb = Images::key_bytes(NI, DKP), vb = Images::value_bytes(NI, p.d_v);
            // 32-channel slices of v (dout) that this CTA has; a pair past them works on what lies there
            const int slices = min(PAIRS / 2, pad_v(p.d_v) / 32 - blk * (PAIRS / 2));
            const int c32 = blk * (PAIRS / 2) * 32;
            auto load_values = [&](uint32_t d, bool image, const char *vimg, int t, uint32_t m) {
                if (image) bulk_load(d, vimg, slices * L::kSlice, m);
                else
                    for (int x = 0; x < slices; ++x) ptx::tma_load_3d(d + x * L::kSlice, &tm_v, c32 + x * 32, head, t, m);
            };
            int done1 = 0, done2 = 0;
            bool ok = true;
            for (int i = 0; i < n_chunks && ok; ++i) {
                const int c = at(i), t = (int)tok0 + c * C;
                const bool image = im.has(t, min(C, len - c * C), p.n_tok);
                const char *img = ws + im.offset + (im.all ? slot0 + c : (int64_t)seq) * rec;
                const char *vimg = img + 2 * p.n_k_heads * kb + (kRev ? p.n_heads + head : head) * vb + (size_t)blk * L::kVal;
                const char *terms = ws + ((slot0 + c) * p.n_heads + head) * terms_bytes(NS);
                {
                    const int s = i % N1;
                    const uint32_t d = base + s * L::kStage1, m = full1(s);
                    if (!(ok = wait_bar(empty1(s), ((i / N1) & 1) ^ 1))) break;
                    ptx::mbar_arrive_tx(m, L::kKey + (kRev ? 0 : slices * L::kSlice) + L::kX + L::kGate);
                    if (image) {
                        bulk_load(d + L::K, img + (p.n_k_heads + kh) * kb, L::kKey, m);
                    } else {
#pragma unroll
                        for (int h = 0; h < DKP / 64; ++h) ptx::tma_load_3d(d + L::K + h * kHalf, &tm_k, h * 64, kh, t, m);
                    }
                    if (!kRev) load_values(d + L::V, image, vimg, t, m);
                    bulk_load(d + L::X, terms, L::kX, m);
                    bulk_load(d + L::Gate1, terms + 2 * NS * kTri, L::kGate, m);
                    ++done1;
                }
                if constexpr (N2 > 0) {
                    const int s = i % N2;
                    const uint32_t d = base + L::Ring2 + s * L::kStage2, m = full2(s);
                    if (!(ok = wait_bar(empty2(s), ((i / N2) & 1) ^ 1))) break;
                    ptx::mbar_arrive_tx(m, L::kKey + (kRev ? slices * L::kSlice : 0) + L::kP + L::kGate);
                    if (image) {
                        bulk_load(d + L::Q, img + kh * kb, L::kKey, m);
                    } else {
#pragma unroll
                        for (int h = 0; h < DKP / 64; ++h) ptx::tma_load_3d(d + L::Q + h * kHalf, &tm_q, h * 64, kh, t, m);
                    }
                    if (kRev) load_values(d + L::dO, image, vimg, t, m);
                    bulk_load(d + L::P, terms + NS * kTri, L::kP, m);
                    bulk_load(d + L::Gate2, terms + 2 * NS * kTri, L::kGate, m);
                    ++done2;
                }
            }
            if (!ok) {  // nothing may land in shared memory after the CTA has gone
                for (int i = max(0, done1 - N1); i < done1; ++i) drain_bar(full1(i % N1), (i / N1) & 1);
                if constexpr (N2 > 0)
                    for (int i = max(0, done2 - N2); i < done2; ++i) drain_bar(full2(i % N2), (i / N2) & 1);
            }
        }
    } else if (warp < 2 * PAIRS) {
        // ------------------------------------------------ state
        // A failed wait ends no warp of a pair before the other (their barriers would hang): the
        // step goes on with what is there, and with the flag set no later wait waits.
        constexpr int kBlk = 512;                      // a plane of a 16 x 16 block
        constexpr int kSP = KX * kBlk, kUP = 4 * kBlk;  // plane strides of Sx and of Ux, Uo
        // In the triangular product the first warp's tokens feed both halves: tokens 0..31
        // forward, 32..63 in reverse.
        const bool first = h == (kRev ? 1 : 0);
        const int t0 = 2 * h, o0 = 2 - t0;             // this half's, the other half's first 16-token block
        auto meet = [&]() { ptx::named_sync(1 + w, 64); };
        float S[NT][4];                                // key channels h DKP / 2 ..
        uint32_t sp[NS][KX][4];                        // all key channels as planes, this half's first
        const int c0 = h * (DKP / 2);
        load_state<NT>(S, kRev ? (p.dh_final ? p.dh_final + st_at : nullptr) : (p.h0 ? p.h0 + st_at : nullptr), c0, v0,
                       p.d_k, p.d_v);
        [[maybe_unused]] char *keep = pair + L::Keep;
        // this half's planes of S^T to the pair's buffer, the other half's from it
        auto share_state = [&](int hb) {
            char *sx = pair + L::Sx + hb * L::kSx;
#pragma unroll
            for (int i = 0; i < KX / 2; ++i) {
                uint32_t a[NS][4];
                acc_to_a<NS>(&S[2 * i], a);
                put_block<NS>(sx + (h * (KX / 2) + i) * kBlk, kSP, a);
#pragma unroll
                for (int q = 0; q < NS; ++q)
#pragma unroll
                    for (int x = 0; x < 4; ++x) sp[q][i][x] = a[q][x];
            }
            meet();
#pragma unroll
            for (int i = 0; i < KX / 2; ++i) {
                uint32_t a[NS][4];
                get_block<NS>(sx + ((1 - h) * (KX / 2) + i) * kBlk, kSP, a);
#pragma unroll
                for (int q = 0; q < NS; ++q)
#pragma unroll
                    for (int x = 0; x < 4; ++x) sp[q][KX / 2 + i][x] = a[q][x];
            }
        };
        if (n_chunks > 0) share_state(0);
        bool ready = false;  // asked ahead of time: the answer's latency hides behind the update of S
        for (int i = 0; i < n_chunks; ++i) {
            const int c = at(i), s1 = i % N1, hb = i % NH;
            const uint32_t s = base + s1 * L::kStage1;
            const float *gate = reinterpret_cast<const float *>(smem + s1 * L::kStage1 + L::Gate1);
            char *rec = ws + scan_offset(p.n_tok, p.n_seq, p.n_heads, NS) +
                        ((slot0 + c) * p.n_heads + head) * scan_bytes(NS, DKP, p.d_v) +
                        ((v0 >> 4) * 2 + kRev) * scan_part(NS, DKP);
            if (!ready) wait_bar(full1(s1), (i / N1) & 1);
            if (kRev && kHelp) wait_bar(hfull(hb), (i / NH) & 1);
            [[maybe_unused]] const int s2 = N2 > 0 ? i % (N2 > 0 ? N2 : 1) : 0;
            [[maybe_unused]] const uint32_t r2 = base + L::Ring2 + s2 * L::kStage2;
            if (!kHelp && N2 > 0 && kRev) wait_bar(full2(s2), (i / (N2 > 0 ? N2 : 1)) & 1);
            __syncwarp();

            // this half's tokens: forward Y^T, then beta Z^T; in reverse dU^T
            uint32_t z[2][NS][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int tb = t0 + b;
                float y[2][4];
                state_times_keys<NI, NS, DKP>(sp, s + L::K, h, tb * 16, y);
                if (!kRev) {  // beta Z^T = beta (V^T - gamma Y^T)
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll
                    for (int q = 0; q < NI; ++q) {
                        uint32_t x[4];
                        ptx::ldsm_x4_t(s + L::V + (w >> 1) * L::kSlice + q * C * 64 +
                                           tile_off<64>(tb * 16 + (lane >> 4) * 8 + (lane & 7), (w & 1) * 16 + ((lane >> 3) & 1) * 8),
                                       x[0], x[1], x[2], x[3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[2 * j] += lo_f(x[j]);
                            v[2 * j + 1] += hi_f(x[j]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int t = tb * 16 + n * 8 + tq * 2;
                        const float2 ga = *reinterpret_cast<const float2 *>(gate + t);
                        const float2 be = *reinterpret_cast<const float2 *>(gate + 2 * C + t);
                        y[n][0] = be.x * fmaf(-ga.x, y[n][0], v[4 * n]);
                        y[n][1] = be.y * fmaf(-ga.y, y[n][1], v[4 * n + 1]);
                        y[n][2] = be.x * fmaf(-ga.x, y[n][2], v[4 * n + 2]);
                        y[n][3] = be.y * fmaf(-ga.y, y[n][3], v[4 * n + 3]);
                    }
                } else {      // dU^T = delta (dS1^T K^T) + dO^T P
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int t = 2 * tb + n;
                        const float2 de = *reinterpret_cast<const float2 *>(gate + C + t * 8 + tq * 2);
                        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (kHelp) x = *reinterpret_cast<const float4 *>(pair + L::Hand + L::kHandG + (t * 32 + lane) * 16);
                        y[n][0] = fmaf(de.x, y[n][0], x.x);
                        y[n][1] = fmaf(de.y, y[n][1], x.y);
                        y[n][2] = fmaf(de.x, y[n][2], x.z);
                        y[n][3] = fmaf(de.y, y[n][3], x.w);
                    }
                    if constexpr (kRev && !kHelp)
#pragma unroll
                        for (int kx = 0; kx < 4; ++kx)
                            if (kx >= tb) {
                                uint32_t f[NI][4];
                                frag_dout<NI>(r2 + L::dO + (w >> 1) * L::kSlice, kx, w & 1, f);
                                add_dout_p<NI, NS>(f, r2 + L::P + tri_block(kx, tb), y);
                            }
                }
                acc_to_a<NS>(y, z[b]);
            }
            if constexpr (!kOut && L::kKeep > 0) {  // this half of S0 (or dS1) to the staging, once the
                if (h == 0 && lane == 0) ptx::bulk_wait_read0();  // last step's record has been read
                meet();
#pragma unroll
                for (int q = 0; q < NS; ++q)
#pragma unroll
                    for (int x = 0; x < KX / 2; ++x)
                        store_block(ptx::smem_u32(keep) + q * L::kKeepP +
                                        state_half(c0 + x * 16) +
                                        tile_off<128>(lane & 15, ((c0 + x * 16) & 63) + (lane >> 4) * 8), sp[q][x]);
            }
            // U^T = (beta Z)^T X^T (X lower triangular), in reverse E^T = dU^T X: each half's diagonal
            // block by its own warp; the block between the halves by the second warp, which gets
            // the first one's planes (it would otherwise wait for that product and its own finish)
            if (first)
#pragma unroll
                for (int b = 0; b < 2; ++b) put_block<NS>(pair + L::Zx + b * kBlk, 2 * kBlk, z[b]);
            float u[4][4];
            zero<4>(u);
            if (first) meet();
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    if (kRev ? n <= b : n >= b)
                        add_times_x<NS, kRev>(z[b], s + L::X, t0 + b, t0 + n, &u[2 * n]);
            if (!first) {
                meet();
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t a[NS][4];
                    get_block<NS>(pair + L::Zx + b * kBlk, 2 * kBlk, a);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
                        add_times_x<NS, kRev>(a, s + L::X, o0 + b, t0 + n, &u[2 * n]);
                }
            }
            auto finish = [&]() {  // u complete: to the output or the record; scaled, to the pair
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t a[NS][4];
                    if constexpr (!kOut) acc_to_a<NS>(&u[2 * b], a);
                    if constexpr (kOut) {  // in fp32: the output warps, which have the time, split it
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            *reinterpret_cast<float4 *>(pair + L::Uo + hb * L::kUo + ((2 * (t0 + b) + n) * 32 + lane) * 16) =
                                make_float4(u[2 * b + n][0], u[2 * b + n][1], u[2 * b + n][2], u[2 * b + n][3]);
                    } else if constexpr (L::kKeep > 0) {
#pragma unroll
                        for (int q = 0; q < NS; ++q)
                            store_block(ptx::smem_u32(keep) + q * L::kKeepP + L::kKeepV +
                                            tile_off<128>(lane & 15, (t0 + b) * 16 + (lane >> 4) * 8), a[q]);
                    } else {  // straight to the record
#pragma unroll
                        for (int q = 0; q < NS; ++q)
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                *reinterpret_cast<uint32_t *>(rec + q * L::kKeepP + L::kKeepV +
                                                              tile_off<128>(gr + (y & 1) * 8, (t0 + b) * 16 + (y >> 1) * 8 + tq * 2)) = a[q][y];
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {  // delta U, in reverse -gamma beta E
                        const int t = (t0 + b) * 16 + n * 8 + tq * 2;
                        float2 f = *reinterpret_cast<const float2 *>(gate + (kRev ? 0 : C) + t);
                        if (kRev) {
                            const float2 be = *reinterpret_cast<const float2 *>(gate + 2 * C + t);
                            f.x *= -be.x;
                            f.y *= -be.y;
                        }
                        float *x = u[2 * b + n];
                        x[0] *= f.x; x[1] *= f.y; x[2] *= f.x; x[3] *= f.y;
                    }
                    acc_to_a<NS>(&u[2 * b], z[b]);
                    put_block<NS>(pair + L::Ux + (t0 + b) * kBlk, kUP, z[b]);
                }
                if (kOut) warp_arrive(hfull(hb));
            };
            // S = Gamma S (+ G = (s gamma dO)^T Q, in reverse) while the other warp finishes its half
            const float whole = gate[3 * C];
            auto decay = [&]() {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (kRev && kHelp) x = *reinterpret_cast<const float4 *>(pair + L::Hand + ((h * NT + n) * 32 + lane) * 16);
                    S[n][0] = fmaf(whole, S[n][0], x.x);
                    S[n][1] = fmaf(whole, S[n][1], x.y);
                    S[n][2] = fmaf(whole, S[n][2], x.z);
                    S[n][3] = fmaf(whole, S[n][3], x.w);
                }
                if (kRev && kHelp) warp_arrive(hempty(hb));
                if constexpr (kRev && !kHelp) {
#pragma unroll
                    for (int kx = 0; kx < 4; ++kx) {
                        uint32_t f[NI][4], d[NS][4];
                        frag_dout<NI>(r2 + L::dO + (w >> 1) * L::kSlice, kx, w & 1, f);
                        scale_dout<NI, NS>(f, gate, scale, kx, d);
                        add_values_keys<NI, NS, DKP>(d, r2 + L::Q, kx * 16, c0, S);
                    }
                    warp_arrive(empty2(s2));
                }
            };
            finish();
            decay();
            if (first) {  // its own tokens' share of S while the second warp is not done
#pragma unroll
                for (int b = 0; b < 2; ++b) add_values_keys<NI, NS, DKP>(z[b], s + L::K, (t0 + b) * 16, c0, S);
                meet();
            } else {
                meet();
#pragma unroll
                for (int b = 0; b < 2; ++b) add_values_keys<NI, NS, DKP>(z[b], s + L::K, (t0 + b) * 16, c0, S);
            }
            bool drained = true;
            if (kOut && i + 1 >= NH) drained = test_bar(hempty((i + 1) % NH), ((i + 1 - NH) / NH) & 1);
            ready = N1 > 1 && test_bar(full1((i + 1) % N1), ((i + 1) / N1) & 1);
#pragma unroll
            for (int b = 0; b < 2; ++b) {  // the other half's tokens
                uint32_t a[NS][4];
                get_block<NS>(pair + L::Ux + (o0 + b) * kBlk, kUP, a);
                add_values_keys<NI, NS, DKP>(a, s + L::K, (o0 + b) * 16, c0, S);
            }
            warp_arrive(empty1(s1));
            if constexpr (!kOut && L::kKeep == 0) {  // this half of S0 (or dS1), straight to the record
#pragma unroll
                for (int q = 0; q < NS; ++q)
#pragma unroll
                    for (int x = 0; x < KX / 2; ++x)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            *reinterpret_cast<uint32_t *>(rec + q * L::kKeepP + state_half(c0 + x * 16) +
                                                          tile_off<128>(gr + (y & 1) * 8, ((c0 + x * 16) & 63) + (y >> 1) * 8 + tq * 2)) = sp[q][x][y];
            }
            if constexpr (L::kKeep > 0) ptx::fence_proxy_async();
            if (!drained)  // the output that read the next step's buffers is done
                wait_bar(hempty((i + 1) % NH), ((i + 1 - NH) / NH) & 1);
            __syncwarp();
            share_state((i + 1) % NH);
            if constexpr (L::kKeep > 0) {
                // both halves are staged (the barrier in share_state): one lane sends the record
                if (h == 0 && lane == 0 && v0 < pad_v(p.d_v)) {
                    bulk_store(rec, ptx::smem_u32(keep), L::kKeep);
                    ptx::bulk_commit();
                }
            }
        }
        if (L::kKeep > 0 && h == 0 && lane == 0) bulk_wait0();
        float *end = kRev ? p.dh0 : kOut ? p.h_final : nullptr;
        if (end) store_state<NT>(S, end + st_at, c0, v0, p.d_k, p.d_v);
    } else if constexpr (kOut) {
        // ------------------------------------------------ output: O = s gamma Q S0 + (s P) U, half h
        for (int i = 0; i < n_chunks; ++i) {
            const int s2 = i % N2, hb = i % NH;
            const uint32_t s = base + L::Ring2 + s2 * L::kStage2;
            const float *gate = reinterpret_cast<const float *>(smem + L::Ring2 + s2 * L::kStage2 + L::Gate2);
            if (!warp_wait(full2(s2), (i / N2) & 1)) break;
            if (!warp_wait(hfull(hb), (i / NH) & 1)) break;
            float o[2][2][4];
            zero<4>(&o[0][0]);
#pragma unroll
            for (int kx = 0; kx < KX; ++kx) {
                uint32_t a[NS][4];
                get_block<NS>(pair + L::Sx + hb * L::kSx + kx * 512, KX * 512, a);
                add_queries<NI, NS, DKP>(a, s + L::Q, h, kx, o);
            }
            scale_output(o, gate, scale, h);
            add_p_values<NS>(pair + L::Uo + hb * L::kUo, s + L::P, h, o);
            warp_arrive(hempty(hb));
            warp_arrive(empty2(s2));
            store_output(static_cast<T *>(p.out), o, i * C, h, v0, tok0, len, head, p, wide_out);
        }
    } else if constexpr (kRev && kHelp) {
        // ------------------------------------------------ G^T = (s gamma dO)^T Q, key channels of half
        // h, and dO^T P, tokens of half h
        for (int i = 0; i < n_chunks; ++i) {
            const int s2 = i % N2, hb = i % NH;
            const uint32_t s = base + L::Ring2 + s2 * L::kStage2;
            const float *gate = reinterpret_cast<const float *>(smem + L::Ring2 + s2 * L::kStage2 + L::Gate2);
            if (!warp_wait(full2(s2), (i / N2) & 1)) break;
            float y[4][4], G[NT][4];
            zero<4>(y);
            zero<NT>(G);
#pragma unroll
            for (int kx = 0; kx < 4; ++kx) {
                uint32_t a[NI][4], d[NS][4];
                frag_dout<NI>(s + L::dO, kx, w, a);
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    if (2 * h + n <= kx) add_dout_p<NI, NS>(a, s + L::P + tri_block(kx, 2 * h + n), &y[2 * n]);
                scale_dout<NI, NS>(a, gate, scale, kx, d);
                add_values_keys<NI, NS, DKP>(d, s + L::Q, kx * 16, h * (DKP / 2), G);
            }
            warp_arrive(empty2(s2));
            if (!warp_wait(hempty(hb), ((i / NH) & 1) ^ 1)) break;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<float4 *>(pair + L::Hand + ((h * NT + n) * 32 + lane) * 16) = make_float4(G[n][0], G[n][1], G[n][2], G[n][3]);
#pragma unroll
            for (int n = 0; n < 4; ++n)
                *reinterpret_cast<float4 *>(pair + L::Hand + L::kHandG + ((4 * h + n) * 32 + lane) * 16) =
                    make_float4(y[n][0], y[n][1], y[n][2], y[n][3]);
            warp_arrive(hfull(hb));
        }
    }
    __syncthreads();  // the barriers outlive every wait
}

inline cudaError_t read_flags(unsigned int *flags, bool reset, cudaStream_t stream) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(flags, g_gdr_flags, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    if (reset) {
        static const unsigned int none = 0;
        e = cudaMemcpyToSymbolAsync(g_gdr_flags, &none, sizeof(none), 0, cudaMemcpyHostToDevice, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaStreamSynchronize(stream);
}

}  // namespace gdr
}  // namespace kda
