// Shared by the kernels of the gated delta rule with one decay per head (kda_gdr_fwd.cu,
// kda_gdr_bwd.cu): sizes, workspace layout, operand tiles and warp-level products.
// Internal; not part of the C ABI.
//
// Precision. Every product runs on bf16 tensor-core operations with fp32 accumulation (mma.sync;
// tcgen05 where a chain of dependent products does not wait for it). An operand that is not a
// bf16 input is carried as a sum of bf16 planes (hi + lo, or hi + mid + lo), so that the fp32
// results (states, gate and beta gradients) keep about 2^-17 of relative error per operand for
// bf16 inputs and 2^-24 for fp32 inputs. NI = planes of an input tile (1: bf16, 3: fp32), NS =
// planes of an intermediate (2 or 3); a product of plane i with plane j is formed only where
// i + j < NS (the rest is below the accumulator's rounding of the sum). What reaches only a bf16
// result is carried in NS planes as well, S0 and P in O, B and F in dQ and dK: in one, the error of O
// is 2.5e-3 and that of dQ and dK 2.2e-3 where their own rounding is 1.7e-3.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_ptx.h"

namespace kda {
namespace gdr {

constexpr int C = 64;           // tokens of a chunk
// A chunk's 64 x 64 lower triangular tile as its ten 16 x 16 blocks on and below the diagonal,
// row after row of blocks, a block's rows of 32 bytes swizzled
constexpr int kTri = 10 * 512;  // bytes of one bf16 plane
__host__ __device__ constexpr int tri_block(int I, int J) { return (I * (I + 1) / 2 + J) * 512; }
constexpr float kGFloor = -200.f;

// ---------------------------------------------------------------- workspace
// Chunk c of sequence n lives in slot (cu[n] / 64) + n + c: distinct over all chunks and
// below n_tok / 64 + n_seq, without a pass over the lengths on the host.
__host__ __device__ __forceinline__ int64_t n_slots(int64_t n_tok, int64_t n_seq) {
    return n_tok / C + n_seq;
}
__device__ __forceinline__ int64_t slot_base(const int32_t *cu, int n) {
    return (int64_t)(cu[n] >> 6) + n;
}

// Dependent launches: the kernel starts while the one before it on the stream drains, and
// waits here for that one's results.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, const A &...args) {
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

struct Chunk {
    int seq, len;      // len = 0: an unused slot
    int64_t t0;
};
// the chunk in a slot
__device__ __forceinline__ Chunk find_chunk(const int32_t *cu, int n_seq, int64_t slot) {
    int lo = 0, hi = n_seq - 1;  // largest n with slot_base(n) <= slot
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (slot_base(cu, mid) <= slot) lo = mid; else hi = mid - 1;
    }
    const int64_t t0 = cu[lo] + (slot - slot_base(cu, lo)) * C;
    const int64_t left = cu[lo + 1] - t0;
    return {lo, left <= 0 ? 0 : left < C ? (int)left : C, t0};
}

// Per (slot, value head): X and P (NS triangular planes each) and the gate vectors gamma, delta, beta,
// Gamma (repeated) and the running sum of g log2(e) as pairs of floats. The chains read the first four.
constexpr int kGateFloats = 6 * C, kChainGates = 4 * C;
__host__ __device__ constexpr size_t terms_bytes(int ns) {
    return (size_t)2 * ns * kTri + kGateFloats * 4;
}

// Per (slot, value head) of the backward pass, behind the terms: for each 16 value channels (of
// d_v padded to a multiple of 32) the forward chain's part, then the reverse chain's. A part is
// NS planes of S0^T (16 x d_k padded to DKP) and U^T (16 x 64), or of dS1^T and E^T: DKP / 64 + 1
// tiles of 16 rows of 128 bytes in the 128-byte swizzle, which tcgen05 reads as one MN-major
// operand. A chain writes a part in one copy and the local gradients read a block in one.
__host__ __device__ __forceinline__ constexpr int pad_v(int d_v) { return (d_v + 31) & ~31; }
__host__ __device__ constexpr int scan_part(int ns, int dkp) { return ns * 16 * (dkp + C) * 2; }
__host__ __device__ __forceinline__ size_t scan_bytes(int ns, int dkp, int d_v) {
    return (size_t)(pad_v(d_v) / 16) * 2 * scan_part(ns, dkp);
}
__host__ __device__ __forceinline__ size_t scan_offset(int64_t n_tok, int64_t n_seq, int64_t n_heads, int ns) {
    return (size_t)n_slots(n_tok, n_seq) * n_heads * terms_bytes(ns);
}

// Tile images of q, k (per key head), v and, for the backward pass, dout (per value head) of
// the chunks that a tensor copy cannot fetch: the last, partial chunk of a sequence that
// another one follows (rows past its end must read as zero, not as the next sequence; past
// the last token the copy itself fills in zeros), and every chunk of inputs that are fp32 or
// not 16-byte aligned. Indexed by sequence when only partial chunks need one, else by slot.
struct Images {
    bool all;           // every chunk has an image
    __device__ bool has(int64_t t0, int len, int64_t n_tok) const { return all || (len < C && t0 + len < n_tok); }
    size_t offset;      // of the first, in the workspace
    __host__ __device__ static size_t key_bytes(int ni, int dkp) { return (size_t)ni * C * dkp * 2; }
    __host__ __device__ static size_t value_bytes(int ni, int d_v) { return (size_t)ni * pad_v(d_v) * C * 2; }
    // one index: q and k of every key head, then v (and dout) of every value head
    __host__ __device__ static size_t record(int ni, int dkp, int d_v, int hk, int hv, int values) {
        return 2 * hk * key_bytes(ni, dkp) + (size_t)values * hv * value_bytes(ni, d_v);
    }
};

// ---------------------------------------------------------------- tiles
// A tile of bf16 rows of RB bytes, 16-byte groups XOR-swizzled so that ldmatrix reads eight
// rows of one column group without bank conflicts.
template <int RB>
__device__ __forceinline__ uint32_t tile_off(int row, int col) {
    constexpr int groups = RB / 16;
    const int g = col >> 3;
    int x;
    if constexpr (RB >= 128) x = row & 7;
    else x = (row / (128 / RB)) & (groups - 1);
    return row * RB + ((g ^ x) << 4) + (col & 7) * 2;
}

// operand fragments of one 16 x 16 block of a tile whose stored rows are m (A), n (B) or the
// contraction index (the _t forms)
template <int RB>
__device__ __forceinline__ void frag_a(uint32_t base, int m0, int k0, uint32_t *a) {
    const int l = threadIdx.x & 31;
    ptx::ldsm_x4(base + tile_off<RB>(m0 + (l & 15), k0 + (l >> 4) * 8), a[0], a[1], a[2], a[3]);
}
template <int RB>
__device__ __forceinline__ void frag_a_t(uint32_t base, int k0, int m0, uint32_t *a) {
    const int l = threadIdx.x & 31;
    ptx::ldsm_x4_t(base + tile_off<RB>(k0 + (l >> 4) * 8 + (l & 7), m0 + ((l >> 3) & 1) * 8),
                   a[0], a[1], a[2], a[3]);
}
// b[0..1]: columns n0..n0+7, b[2..3]: columns n0+8..n0+15
template <int RB>
__device__ __forceinline__ void frag_b(uint32_t base, int n0, int k0, uint32_t *b) {
    const int l = threadIdx.x & 31;
    ptx::ldsm_x4(base + tile_off<RB>(n0 + (l >> 4) * 8 + (l & 7), k0 + ((l >> 3) & 1) * 8),
                 b[0], b[1], b[2], b[3]);
}
template <int RB>
__device__ __forceinline__ void frag_b_t(uint32_t base, int k0, int n0, uint32_t *b) {
    const int l = threadIdx.x & 31;
    ptx::ldsm_x4_t(base + tile_off<RB>(k0 + (l & 15), n0 + (l >> 4) * 8), b[0], b[1], b[2], b[3]);
}

// A tile of 64 tokens x DKP key channels: column halves of 64, each 64 rows of 128 bytes in
// the tensor copy's 128-byte swizzle
constexpr int kHalf = C * 128;
__device__ __forceinline__ int key_off(int row, int col) { return (col >> 6) * kHalf + tile_off<128>(row, col & 63); }
__device__ __forceinline__ void key_a(uint32_t base, int m0, int k0, uint32_t *a) {
    frag_a<128>(base + (k0 >> 6) * kHalf, m0, k0 & 63, a);
}
__device__ __forceinline__ void key_b(uint32_t base, int n0, int k0, uint32_t *b) {
    frag_b<128>(base + (k0 >> 6) * kHalf, n0, k0 & 63, b);
}
__device__ __forceinline__ void key_b_t(uint32_t base, int k0, int n0, uint32_t *b) {
    frag_b_t<128>(base + (n0 >> 6) * kHalf, k0, n0 & 63, b);
}

// Byte offset of the tile of key channel c in a plane of a part; U^T or E^T is the tile after the
// last. The rest of the offset is tile_off<128>(value channel, c % 64).
__device__ __forceinline__ int state_half(int c) { return (c >> 6) * 2048; }

// A sum carried as two floats (the fp64 pipe of this part is narrow), each addition's error by
// Knuth's two-sum.
struct Two { float hi, lo; };
__device__ __forceinline__ Two add(Two x, Two y) {
    const float s = x.hi + y.hi, t = s - x.hi;
    const float e = (x.hi - (s - t)) + (y.hi - t) + (x.lo + y.lo);
    const float hi = s + e;
    return {hi, e - (hi - s)};
}
// acc (two neighbouring 16 x 8 tiles) += A B from planes a, b: the products of planes i + j < LIM.
// With three planes the tensor cores' own sums show: they drop bits of every addend below the
// running sum's last place. The smallest products are then summed first, in accumulators that
// start at zero, and only their sum meets acc, rounded to nearest.
template <int NA, int NB, int LIM>
__device__ __forceinline__ void product(float (*acc)[4], const uint32_t (*a)[4], const uint32_t (*b)[4]) {
    if constexpr (LIM == 3) {
        float t[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[0][i] = t[1][i] = 0.f;
#pragma unroll
        for (int level = LIM - 1; level >= 0; --level)
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                if (i > level || level - i >= NB) continue;
                ptx::mma16816(t[0], a[i], b[level - i][0], b[level - i][1]);
                ptx::mma16816(t[1], a[i], b[level - i][2], b[level - i][3]);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[0][i] += t[0][i];
            acc[1][i] += t[1][i];
        }
    } else {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                if (i + j >= LIM) continue;
                ptx::mma16816(acc[0], a[i], b[j][0], b[j][1]);
                ptx::mma16816(acc[1], a[i], b[j][2], b[j][3]);
            }
    }
}

// 2^x (0 below the normal range)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two fp32 values as NP packed planes whose sum is the value
template <int NP>
__device__ __forceinline__ void split2(float x, float y, uint32_t *p) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const uint32_t w = ptx::pack_bf16(x, y);
        p[i] = w;
        if (i + 1 < NP) {
            x -= __uint_as_float(w << 16);
            y -= __uint_as_float(w & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// acc tiles t0 = d[0], t1 = d[1] (columns 0..7 and 8..15 of a 16 x 16 block): as the A
// operand whose contraction index is the block's column; plane p in a[p][0..3]
template <int NP>
__device__ __forceinline__ void acc_to_a(const float (*d)[4], uint32_t (*a)[4]) {
    uint32_t w[NP];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float *t = d[i >> 1];
        split2<NP>(t[(i & 1) * 2], t[(i & 1) * 2 + 1], w);
#pragma unroll
        for (int p = 0; p < NP; ++p) a[p][i] = w[p];
    }
}

// ---------------------------------------------------------------- loading inputs
template <typename T> struct InputPlanes;
template <> struct InputPlanes<__nv_bfloat16> { static constexpr int N = 1; };
template <> struct InputPlanes<float> { static constexpr int N = 3; };

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void st_shared_16(uint32_t a, const uint32_t *w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]) : "memory");
}

// C rows of RB / 2 columns from src (rows `stride` elements apart) into the tile at `dst`
// (planes `plane` bytes apart); rows >= rows and columns >= cols read as zero. vec: the rows
// are 16-byte aligned and cols fills whole 16-byte groups (then bf16 goes by cp.async).
template <typename T, int RB>
__device__ __forceinline__ void load_tile(uint32_t dst, uint32_t plane, const T *src, int64_t stride,
                                          int rows, int cols, bool vec, int tid, int nthreads) {
    constexpr int groups = RB / 16;
    for (int i = tid; i < C * groups; i += nthreads) {
        const int r = i / groups, c = (i % groups) * 8;
        const uint32_t at = dst + tile_off<RB>(r, c);
        const bool in = r < rows && c < cols;
        const T *p = src + (in ? r * stride + c : 0);
        if constexpr (sizeof(T) == 2) {
            if (vec) {
                cp_async_16(at, p, in ? 16 : 0);
                continue;
            }
            uint32_t w[4] = {0, 0, 0, 0};
            if (in) {
                const uint16_t *e = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < cols) w[j >> 1] |= (uint32_t)e[j] << (16 * (j & 1));
            }
            st_shared_16(at, w);
        } else {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.f;
            if (in) {
                const float *e = reinterpret_cast<const float *>(p);
                if (vec && c + 8 <= cols) {
                    const float4 u = *reinterpret_cast<const float4 *>(e);
                    const float4 v = *reinterpret_cast<const float4 *>(e + 4);
                    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
                    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (c + j < cols) x[j] = e[j];
                }
            }
            uint32_t w[3][4], s[3];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                split2<3>(x[2 * j], x[2 * j + 1], s);
                w[0][j] = s[0]; w[1][j] = s[1]; w[2][j] = s[2];
            }
#pragma unroll
            for (int q = 0; q < 3; ++q) st_shared_16(at + q * plane, w[q]);
        }
    }
}
// the key tile of a chunk (planes C * DKP * 2 bytes apart)
template <typename T, int DKP>
__device__ __forceinline__ void load_key_tile(uint32_t dst, const T *src, int64_t stride, int rows, int cols,
                                              bool vec, int tid, int nthreads) {
#pragma unroll
    for (int h = 0; h < DKP / 64; ++h)
        load_tile<T, 128>(dst + h * kHalf, C * DKP * 2, src + h * 64, stride, rows, cols - h * 64, vec, tid, nthreads);
}
// The images of `heads` neighbouring value tiles of a chunk (vb bytes apart): slices of 32
// channels, each NI planes of 64 rows of 64 bytes in the tensor copy's 64-byte swizzle.
template <typename T>
__device__ __forceinline__ void write_value_images(char *dst, size_t vb, const T *src, int64_t stride, int heads,
                                                   int rows, int cols, int tid, int nthreads) {
    constexpr int NI = InputPlanes<T>::N, plane = C * 64;
    const int per = pad_v(cols) / 32 * C * 4;
    const bool vec = sizeof(T) == 2 && cols % 8 == 0 && ((uintptr_t)src & 15) == 0 && (stride & 7) == 0;
#pragma unroll 4
    for (int i = tid; i < heads * per; i += nthreads) {
        const int head = i / per, k = i - head * per;
        const int sl = k / (C * 4), r = (k >> 2) % C, c = (k & 3) * 8, col = sl * 32 + c;
        const T *p = src + r * stride + head * cols + col;
        char *at = dst + head * vb + sl * NI * plane + tile_off<64>(r, c);
        const bool in = r < rows && col < cols;
        if (vec) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in) x = *reinterpret_cast<const uint4 *>(p);
            *reinterpret_cast<uint4 *>(at) = x;
            continue;
        }
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = in && col + j < cols ? (float)p[j] : 0.f;
        uint32_t w[NI][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t s[NI];
            split2<NI>(x[2 * j], x[2 * j + 1], s);
#pragma unroll
            for (int q = 0; q < NI; ++q) w[q][j] = s[q];
        }
#pragma unroll
        for (int q = 0; q < NI; ++q)
            *reinterpret_cast<uint4 *>(at + q * plane) = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
    }
}
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
// two neighbouring elements; wide: p is aligned to both
__device__ __forceinline__ void put2(float *p, float x, float y, bool wide, bool second) {
    if (wide) *reinterpret_cast<float2 *>(p) = make_float2(x, y);
    else { p[0] = x; if (second) p[1] = y; }
}
__device__ __forceinline__ void put2(__nv_bfloat16 *p, float x, float y, bool wide, bool second) {
    if (wide) *reinterpret_cast<uint32_t *>(p) = ptx::pack_bf16(x, y);
    else { put(p, x); if (second) put(p + 1, y); }
}

// 16-byte loads of rows of `d` elements at this base and stride
template <typename T>
bool rows_vec(const void *p, int64_t stride, int d) {
    return ((uintptr_t)p & 15u) == 0 && (stride * sizeof(T)) % 16 == 0 && (d * sizeof(T)) % 16 == 0;
}

}  // namespace gdr

// Chunk terms (X, P, gates of every chunk and value head) and the tile images into the
// workspace; `values` = 2 when dout has images too, `ns` planes.
cudaError_t launch_gdr_terms(const GdrArgs &args, gdr::Images images, int values, int ns, cudaStream_t stream);

}  // namespace kda
