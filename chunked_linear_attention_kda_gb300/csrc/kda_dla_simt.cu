// kda_dla_simt.cu -- linear attention with one decay per head for fp32 inputs, without tensor cores,
// forward and backward; the formulas are in kda_dla.h.
//
// Chunks of 64 tokens, all side by side: a launch forms what each chunk adds to the state (and, backward,
// to the state's gradient), a second one walks over every sequence's chunks element by element and
// leaves the state at each chunk's start (the gradient of its end) in their place, a third forms
// every chunk's results. Products are fp32 FMAs on tiles in shared memory, a thread holding 4 rows x 4 or 8
// columns of a 64 x 64 or 64 x 128 result: per step of the contraction 32 FMAs for 9 reads, so that the
// FMA pipe bounds a chunk. (A walk that formed the chunks' sums as it went took 4.8 us a chunk: 1531 tokens
// of 6 heads, 72 x 100, 137 us in all; 47 so, sums 13, walk 11, results 27. 777 tokens of 4 heads, 64 x 40,
// backward: 56 us.)
#include <cuda_bf16.h>

#include "kda_dla.h"

namespace kda {
namespace dla {
namespace {

constexpr int C = 64, kThreads = 256;
constexpr int LW = 68;  // floats between rows of the 64 x 64 pair weights: rows 4 banks apart, as in all tiles
constexpr int kDkBlock = 32;

struct Gates {
    float2 G[C];     // sums of g log2(e) up to and with each token
    float gam[C], del[C];
    Two whole;  // in two parts
};
// by one warp; tokens past the chunk's end have g = 0
__device__ void chunk_gates(const DlaArgs &p, const Chunk &ch, int head, Gates *out) {
    const int lane = threadIdx.x & 31;
    Two s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 2 * lane + i;
        s[i] = decay_exponent(r < ch.len ? p.g[(ch.t0 + r) * p.g_stride + head] : 0.f);
    }
    s[1] = add(s[0], s[1]);
    const Two run = warp_scan(s[1]), total = last_lane(run);
    Two before = up(run, 1);
    if (lane == 0) before = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 2 * lane + i;
        const Two G = i ? run : add(before, s[0]);
        out->G[r] = make_float2(G.hi, G.lo);
        out->gam[r] = exp2_of(G);
        out->del[r] = exp2_between(make_float2(total.hi, total.lo), make_float2(G.hi, G.lo));
    }
    if (lane == 0) {
        const float n = rintf(total.hi);
        out->whole = exp2_parts(n, (total.hi - n) + total.lo);
    }
}

// rows x cols of src into a tile of 64 x W, zeros beyond
template <int W>
__device__ __forceinline__ void load_tile(float *dst, const float *src, int64_t stride, int rows, int cols) {
#pragma unroll 8
    for (int i = threadIdx.x; i < C * W; i += kThreads) {
        const int r = i / W, c = i % W;
        dst[r * (W + 4) + c] = r < rows && c < cols ? src[r * stride + c] : 0.f;
    }
}

// A thread's part of a product: rows 4 tr + i, columns tc + 16 j
__device__ __forceinline__ int tr() { return threadIdx.x >> 4; }
__device__ __forceinline__ int tc() { return threadIdx.x & 15; }
// acc += A B, A (64 x n) and B (n x 16 NJ) by rows; n a multiple of 4
template <int NJ>
__device__ __forceinline__ void mm_nn(float (*acc)[NJ], const float *A, int lda, const float *B, int n) {
    constexpr int LB = 16 * NJ + 4;
    const float *a = A + 4 * tr() * lda, *b = B + tc();
    for (int k = 0; k < n; k += 4) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(a + i * lda + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const float y = b[(k + kk) * LB + 16 * j];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = fmaf((&x[i].x)[kk], y, acc[i][j]);
            }
    }
}
// acc += A B^T, A (64 x n) and B (16 NJ x n) by rows of `ld` floats
template <int NJ>
__device__ __forceinline__ void mm_nt(float (*acc)[NJ], const float *A, const float *B, int ld, int n) {
    const float *a = A + 4 * tr() * ld, *b = B + tc() * ld;
    for (int k = 0; k < n; k += 4) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(a + i * ld + k);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float4 y = *reinterpret_cast<const float4 *>(b + 16 * j * ld + k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i][j] = fmaf(x[i].w, y.w, fmaf(x[i].z, y.z, fmaf(x[i].y, y.y, fmaf(x[i].x, y.x, acc[i][j]))));
        }
    }
}
// acc += A^T B, A (64 x 64, rows LW apart) and B (64 x 16 NJ) by rows
template <int NJ>
__device__ __forceinline__ void mm_tn(float (*acc)[NJ], const float *A, const float *B) {
    constexpr int LB = 16 * NJ + 4;
    const float *a = A + 4 * tr(), *b = B + tc();
#pragma unroll 4
    for (int k = 0; k < C; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(a + k * LW);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float y = b[k * LB + 16 * j];
            acc[0][j] = fmaf(x.x, y, acc[0][j]);
            acc[1][j] = fmaf(x.y, y, acc[1][j]);
            acc[2][j] = fmaf(x.z, y, acc[2][j]);
            acc[3][j] = fmaf(x.w, y, acc[3][j]);
        }
    }
}
template <int NJ>
__device__ __forceinline__ void clear(float (*acc)[NJ]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = 0.f;
}
// rows < rows of a result to `out`, rows `stride` apart
template <int NJ>
__device__ __forceinline__ void store_result(float *out, int64_t stride, const float (*x)[NJ], int rows, int cols) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * tr() + i;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int c = tc() + 16 * j;
            if (r < rows && c < cols) out[r * stride + c] = x[i][j];
        }
    }
}
// over the 16 threads that share rows
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The workspace: [directions][slots][heads] states, as many decays in two parts, then (backward) sums of dg and the
// parts of dq and dk of shared heads.
struct Space {
    size_t state, decays, sums, dq, dk, floats;
};
__host__ __device__ inline Space space(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k, int32_t d_v, bool bwd) {
    const size_t chunks = (size_t)n_slots(n_tok, n_seq) * n_heads, walks = bwd ? 2 : 1;
    Space s;
    s.state = (size_t)d_k * d_v;
    s.decays = walks * chunks * s.state;
    s.sums = s.decays + 2 * walks * chunks;
    s.dq = s.sums + (bwd ? chunks : 0);
    s.dk = s.dq + (bwd && n_heads > n_k_heads ? (size_t)n_tok * n_heads * d_k : 0);
    s.floats = s.dk + (s.dk - s.dq);
    return s;
}
__device__ __forceinline__ Space space_of(const DlaArgs &p, bool bwd) {
    return space(p.n_tok, p.n_seq, p.n_heads, p.n_k_heads, p.d_k, p.d_v, bwd);
}
__device__ __forceinline__ int64_t chunk_at(const DlaArgs &p, int64_t slot, int head, bool rev) {
    return ((rev ? n_slots(p.n_tok, p.n_seq) : 0) + slot) * p.n_heads + head;
}

// ---------------------------------------------------------------- states
// What a chunk adds: one CTA per (chunk, head, 32 key channels; backward also direction)
__global__ void __launch_bounds__(kThreads) dla_simt_add_kernel(const DlaArgs p, bool bwd) {
    __shared__ __align__(16) float ks[C][kDkBlock], vs[C][128];
    __shared__ Gates gate;
    gdr::let_next_kernel_start();
    const int64_t slot = blockIdx.x;
    const Chunk ch = find_chunk(p.cu_seqlens, p.n_seq, slot);
    if (ch.len == 0) return;
    const int head = blockIdx.y, kh = head / (p.n_heads / p.n_k_heads), tid = threadIdx.x;
    const int n_blk = (p.d_k + kDkBlock - 1) / kDkBlock, i0 = blockIdx.z % n_blk * kDkBlock;
    const bool rev = (int)blockIdx.z >= n_blk;
    const int ti = (tid >> 5) * 4, tj = (tid & 31) * 4;
    const float *key = static_cast<const float *>(rev ? p.q : p.k) + ch.t0 * (rev ? p.q_stride : p.k_stride) + (int64_t)kh * p.d_k + i0;
    const int64_t key_stride = rev ? p.q_stride : p.k_stride, val_stride = rev ? (int64_t)p.n_heads * p.d_v : p.v_stride;
    const float *val = static_cast<const float *>(rev ? p.dout : p.v) + ch.t0 * val_stride + (int64_t)head * p.d_v;
    if (tid < 32) chunk_gates(p, ch, head, &gate);
#pragma unroll
    for (int x = 0; x < C * kDkBlock / kThreads; ++x) {
        const int r = (tid + x * kThreads) / kDkBlock, i = tid % kDkBlock;
        ks[r][i] = r < ch.len && i0 + i < p.d_k ? key[r * key_stride + i] : 0.f;
    }
    float vx[C * 128 / kThreads];
#pragma unroll
    for (int x = 0; x < C * 128 / kThreads; ++x) {
        const int r = (tid + x * kThreads) / 128, j = tid % 128;
        vx[x] = r < ch.len && j < p.d_v ? val[r * val_stride + j] : 0.f;
    }
    __syncthreads();
    // the decay goes to the values: one factor a row
#pragma unroll
    for (int x = 0; x < C * 128 / kThreads; ++x) {
        const int r = (tid + x * kThreads) / 128;
        vs[r][tid % 128] = vx[x] * (rev ? p.scale * gate.gam[r] : gate.del[r]);
    }
    __syncthreads();
    float add[4][4];
    clear<4>(add);
#pragma unroll 8
    for (int r = 0; r < C; ++r) {
        const float4 k4 = *reinterpret_cast<const float4 *>(&ks[r][ti]);
        const float4 v4 = *reinterpret_cast<const float4 *>(&vs[r][tj]);
        const float k[4] = {k4.x, k4.y, k4.z, k4.w}, v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) add[i][j] = fmaf(k[i], v[j], add[i][j]);
    }
    const Space s = space_of(p, bwd);
    float *ws = static_cast<float *>(p.workspace);
    const int64_t at = chunk_at(p, slot, head, rev);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + ti + i < p.d_k && tj + j < p.d_v) ws[at * s.state + (int64_t)(i0 + ti + i) * p.d_v + tj + j] = add[i][j];
    if (i0 == 0 && tid == 0) {
        ws[s.decays + 2 * at] = gate.whole.hi;
        ws[s.decays + 2 * at + 1] = gate.whole.lo;
    }
}

// The states at the chunks' starts (reverse: the gradients of their ends) in place of what the chunks
// add, and the sequences' last: one element of a sequence's and head's state a thread
__global__ void __launch_bounds__(kThreads) dla_simt_walk_kernel(const DlaArgs p, bool bwd) {
    constexpr int kAhead = 8;
    gdr::let_next_kernel_start();
    gdr::wait_for_previous_kernel();
    const bool rev = blockIdx.z == 1;
    const int seq = blockIdx.x / p.n_heads, head = blockIdx.x % p.n_heads;
    const Space s = space_of(p, bwd);
    const int64_t i = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    if (i >= (int64_t)s.state) return;
    const int64_t given = ((int64_t)seq * p.n_heads + head) * s.state + i;
    const float *from = rev ? p.dh_final : p.h0;
    float *to = rev ? p.dh0 : p.h_final, *ws = static_cast<float *>(p.workspace);
    const int64_t len = p.cu_seqlens[seq + 1] - p.cu_seqlens[seq];
    const int64_t nc = (len + C - 1) / C, slot0 = slot_base(p.cu_seqlens, seq);
    float x = from ? from[given] : 0.f;
    Factors decays;
    for (int64_t n0 = 0; n0 < nc; n0 += kAhead) {
        float add[kAhead];
        Two decay[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
            if (n0 + e < nc) {
                const int64_t at = chunk_at(p, slot0 + (rev ? nc - 1 - n0 - e : n0 + e), head, rev);
                add[e] = ws[at * s.state + i];
                decay[e] = {ws[s.decays + 2 * at], ws[s.decays + 2 * at + 1]};
            }
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
            if (n0 + e < nc) {
                ws[chunk_at(p, slot0 + (rev ? nc - 1 - n0 - e : n0 + e), head, rev) * s.state + i] = x;
                x = fmaf(decays.next(decay[e]), x, add[e]);
            }
    }
    if (to) to[given] = x;
}

// ---------------------------------------------------------------- output
template <int NK, int NV>
struct OutSmem {
    static constexpr int LK = 16 * NK + 4, LV = 16 * NV + 4;
    float q[C * LK], k[C * LK], v[C * LV], s[16 * NK * LV], w[C * LW];
    Gates gate;
};
template <int NK, int NV>
__device__ __forceinline__ void load_state(float *dst, const float *src, int d_k, int d_v) {
#pragma unroll 8
    for (int i = threadIdx.x; i < 256 * NK * NV; i += kThreads) {
        const int r = i / (16 * NV), c = i % (16 * NV);
        dst[r * (16 * NV + 4) + c] = r < d_k && c < d_v ? src[(int64_t)r * d_v + c] : 0.f;
    }
}
// w = scale e x, x (64 x 64) held 4 rows x 4 columns a thread
__device__ __forceinline__ void weights(float *w, const float (*x)[4], const Gates &gate, float scale) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * tr() + i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = tc() + 16 * j;
            w[r * LW + c] = r >= c ? scale * exp2_between(gate.G[r], gate.G[c]) * x[i][j] : 0.f;
        }
    }
}

template <int NK, int NV>
__global__ void __launch_bounds__(kThreads) dla_simt_out_kernel(const DlaArgs p) {
    using S = OutSmem<NK, NV>;
    extern __shared__ __align__(16) char smem_raw[];
    S &s = *reinterpret_cast<S *>(smem_raw);
    const int64_t slot = blockIdx.x;
    const Chunk ch = find_chunk(p.cu_seqlens, p.n_seq, slot);
    if (ch.len == 0) {
        gdr::wait_for_previous_kernel();
        return;
    }
    const int head = blockIdx.y, kh = head / (p.n_heads / p.n_k_heads);
    load_tile<16 * NK>(s.q, static_cast<const float *>(p.q) + ch.t0 * p.q_stride + (int64_t)kh * p.d_k, p.q_stride, ch.len, p.d_k);
    load_tile<16 * NK>(s.k, static_cast<const float *>(p.k) + ch.t0 * p.k_stride + (int64_t)kh * p.d_k, p.k_stride, ch.len, p.d_k);
    load_tile<16 * NV>(s.v, static_cast<const float *>(p.v) + ch.t0 * p.v_stride + (int64_t)head * p.d_v, p.v_stride, ch.len, p.d_v);
    gdr::wait_for_previous_kernel();
    load_state<NK, NV>(s.s, static_cast<const float *>(p.workspace) + chunk_at(p, slot, head, false) * p.d_k * p.d_v, p.d_k, p.d_v);
    if (threadIdx.x < 32) chunk_gates(p, ch, head, &s.gate);
    __syncthreads();
    const int dk4 = (p.d_k + 3) & ~3;
    float qk[4][4], o[4][NV];
    clear<4>(qk);
    mm_nt<4>(qk, s.q, s.k, S::LK, dk4);
    weights(s.w, qk, s.gate, p.scale);
    clear<NV>(o);
    mm_nn<NV>(o, s.q, S::LK, s.s, dk4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f = p.scale * s.gate.gam[4 * tr() + i];
#pragma unroll
        for (int j = 0; j < NV; ++j) o[i][j] *= f;
    }
    __syncthreads();
    mm_nn<NV>(o, s.w, LW, s.v, C);
    store_result<NV>(static_cast<float *>(p.out) + (ch.t0 * p.n_heads + head) * p.d_v, (int64_t)p.n_heads * p.d_v, o, ch.len, p.d_v);
}

// ---------------------------------------------------------------- gradients
// One CTA per (chunk, value head); the parts of dQ and dK of heads that share a key head are added up by a
// launch of their own, in a fixed order.
template <int NK, int NV>
struct GradSmem {
    static constexpr int LK = 16 * NK + 4, LV = 16 * NV + 4;
    float q[C * LK], k[C * LK], v[C * LV], d[C * LV], s[16 * NK * LV], w[C * LW];
    Gates gate;
    float a[C], b[C], row[C], col[8][C], ss[8];
};

template <int NK, int NV>
__global__ void __launch_bounds__(kThreads) dla_simt_grad_kernel(const DlaArgs p) {
    using S = GradSmem<NK, NV>;
    extern __shared__ __align__(16) char smem_raw[];
    S &s = *reinterpret_cast<S *>(smem_raw);
    const int64_t slot = blockIdx.x;
    const Chunk ch = find_chunk(p.cu_seqlens, p.n_seq, slot);
    const int head = blockIdx.y, group = p.n_heads / p.n_k_heads, kh = head / group;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Space at = space_of(p, true);
    float *ws = static_cast<float *>(p.workspace);
    float *sums = p.dg && p.g_stride == 0 ? ws + at.sums : nullptr;
    gdr::let_next_kernel_start();
    if (ch.len == 0) {
        gdr::wait_for_previous_kernel();
        if (sums && tid == 0) sums[slot * p.n_heads + head] = 0.f;
        return;
    }
    const int dk4 = (p.d_k + 3) & ~3, dv4 = (p.d_v + 3) & ~3;
    const int64_t row = (int64_t)p.n_heads * p.d_v;
    load_tile<16 * NK>(s.q, static_cast<const float *>(p.q) + ch.t0 * p.q_stride + (int64_t)kh * p.d_k, p.q_stride, ch.len, p.d_k);
    load_tile<16 * NK>(s.k, static_cast<const float *>(p.k) + ch.t0 * p.k_stride + (int64_t)kh * p.d_k, p.k_stride, ch.len, p.d_k);
    load_tile<16 * NV>(s.v, static_cast<const float *>(p.v) + ch.t0 * p.v_stride + (int64_t)head * p.d_v, p.v_stride, ch.len, p.d_v);
    load_tile<16 * NV>(s.d, static_cast<const float *>(p.dout) + ch.t0 * row + (int64_t)head * p.d_v, row, ch.len, p.d_v);
    gdr::wait_for_previous_kernel();
    load_state<NK, NV>(s.s, ws + chunk_at(p, slot, head, false) * at.state, p.d_k, p.d_v);
    if (warp == 0) chunk_gates(p, ch, head, &s.gate);
    __syncthreads();
    float dq[4][NK], dk[4][NK], qk[4][4], ov[4][4];
    clear<NK>(dq);
    mm_nt<NK>(dq, s.d, s.s, S::LV, dv4);  // dO S0^T
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * tr() + i;
        const float f = p.scale * s.gate.gam[r];
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            a = fmaf(s.q[r * S::LK + tc() + 16 * j], dq[i][j], a);
            dq[i][j] *= f;
        }
        a = row_sum(a);
        if (tc() == 0) s.a[r] = f * a;
    }
    clear<4>(qk);
    clear<4>(ov);
    mm_nt<4>(qk, s.q, s.k, S::LK, dk4);
    mm_nt<4>(ov, s.d, s.v, S::LV, dv4);
    weights(s.w, ov, s.gate, p.scale);
    // sums of W_rj q_r.k_j below the diagonal
    float col[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * tr() + i;
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = tc() + 16 * j;
            const float y = r > c ? s.w[r * LW + c] * qk[i][j] : 0.f;
            m += y;
            col[j] += y;
        }
        m = row_sum(m);
        if (tc() == 0) s.row[r] = m;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        col[j] += __shfl_xor_sync(0xffffffffu, col[j], 16);
        if (lane < 16) s.col[warp][tc() + 16 * j] = col[j];
    }
    __syncthreads();
    clear<NK>(dk);
    mm_nn<NK>(dq, s.w, LW, s.k, C);
    mm_tn<NK>(dk, s.w, s.q);
    {
        float *part = group > 1 ? ws + at.dq + (ch.t0 * p.n_heads + head) * p.d_k : static_cast<float *>(p.dq) + (ch.t0 * p.n_k_heads + kh) * p.d_k;
        store_result<NK>(part, (int64_t)(group > 1 ? p.n_heads : p.n_k_heads) * p.d_k, dq, ch.len, p.d_k);
    }
    __syncthreads();
    const float *end = ws + chunk_at(p, slot, head, true) * at.state;
    float ss = 0.f;
#pragma unroll 8
    for (int i = tid; i < 256 * NK * NV; i += kThreads) {
        const int r = i / (16 * NV), c = i % (16 * NV);
        const float y = r < p.d_k && c < p.d_v ? end[(int64_t)r * p.d_v + c] : 0.f;
        ss = fmaf(s.s[r * S::LV + c], y, ss);
        s.s[r * S::LV + c] = y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) s.ss[warp] = ss;
    weights(s.w, qk, s.gate, p.scale);
    __syncthreads();
    float x[4][NK], y[4][NV];
    clear<NK>(x);
    mm_nt<NK>(x, s.v, s.s, S::LV, dv4);  // V dS1^T
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * tr() + i;
        const float f = s.gate.del[r];
        float b = 0.f;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            b = fmaf(s.k[r * S::LK + tc() + 16 * j], x[i][j], b);
            dk[i][j] = fmaf(f, x[i][j], dk[i][j]);
        }
        b = row_sum(b);
        if (tc() == 0) s.b[r] = f * b;
    }
    {
        float *part = group > 1 ? ws + at.dk + (ch.t0 * p.n_heads + head) * p.d_k : static_cast<float *>(p.dk) + (ch.t0 * p.n_k_heads + kh) * p.d_k;
        store_result<NK>(part, (int64_t)(group > 1 ? p.n_heads : p.n_k_heads) * p.d_k, dk, ch.len, p.d_k);
    }
    clear<NV>(y);
    mm_nn<NV>(y, s.k, S::LK, s.s, dk4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f = s.gate.del[4 * tr() + i];
#pragma unroll
        for (int j = 0; j < NV; ++j) y[i][j] *= f;
    }
    mm_tn<NV>(y, s.w, s.d);
    store_result<NV>(static_cast<float *>(p.dv) + ch.t0 * row + (int64_t)head * p.d_v, row, y, ch.len, p.d_v);
    if (!p.dg) return;
    __syncthreads();
    if (warp == 0) {  // two tokens a lane, running sums over the chunk
        float whole = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) whole += s.ss[i];
        whole *= s.gate.whole.hi;
        Two a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            float c = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) c += s.col[w][r];
            a[i] = add({s.a[r], 0.f}, add({s.row[r], 0.f}, {-c, 0.f}));
            b[i] = {s.b[r], 0.f};
        }
        const Two ra = warp_scan(add(a[0], a[1])), rb = warp_scan(add(b[0], b[1]));
        const Two total = last_lane(ra);
        Two a0 = up(ra, 1), b0 = up(rb, 1);
        if (lane == 0) a0 = b0 = {0.f, 0.f};
        float both = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            const Two before = i ? add(a0, a[0]) : a0, sb = i ? add(b0, b[0]) : b0;
            const Two sum = add(minus(total, before), add({whole, 0.f}, sb));
            const int64_t t = (ch.t0 + r) * p.g_stride + head;
            if (r < ch.len) {  // nothing passes a decay of 0: what the sums leave there is rounding
                const float d = p.g[t] < kGFloor ? 0.f : sum.hi + sum.lo;
                if (sums) both += d;
                else p.dg[t] = d;
            }
        }
        if (sums) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) both += __shfl_xor_sync(0xffffffffu, both, o);
            if (lane == 0) sums[slot * p.n_heads + head] = both;
        }
    }
}

// dq (blockIdx.y = 0) or dk of a key head: the sum of its value heads' parts
__global__ void __launch_bounds__(kThreads) dla_simt_shared_heads_kernel(const DlaArgs p) {
    gdr::wait_for_previous_kernel();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, group = p.n_heads / p.n_k_heads;
    if (i >= (int64_t)p.cu_seqlens[p.n_seq] * p.n_k_heads * p.d_k) return;
    const Space at = space_of(p, true);
    const float *from = static_cast<const float *>(p.workspace) + (blockIdx.y ? at.dk : at.dq) + i / p.d_k * group * p.d_k + i % p.d_k;
    float x = 0.f;
    for (int64_t h = 0; h < group; ++h) x += from[h * p.d_k];
    static_cast<float *>(blockIdx.y ? p.dk : p.dq)[i] = x;
}

// dg[head] = the chunks' sums added up, one CTA per head, in a fixed order
__global__ void __launch_bounds__(kThreads) dla_sum_decay_kernel(const float *sums, int64_t rows, int heads, float *dg) {
    __shared__ float part[kThreads / 32];
    float x = 0.f;
    for (int64_t i = threadIdx.x; i < rows; i += kThreads) x += sums[i * heads + blockIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
        x = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) x += part[i];
        dg[blockIdx.x] = x;
    }
}

template <int NK, int NV>
cudaError_t results(const DlaArgs &p, bool bwd, cudaStream_t stream) {
    const dim3 grid((unsigned)n_slots(p.n_tok, p.n_seq), p.n_heads);
    return bwd ? gdr::launch_dependent(dla_simt_grad_kernel<NK, NV>, grid, kThreads, sizeof(GradSmem<NK, NV>), stream, p)
               : gdr::launch_dependent(dla_simt_out_kernel<NK, NV>, grid, kThreads, sizeof(OutSmem<NK, NV>), stream, p);
}

}  // namespace

cudaError_t launch_dla_sum_decay(const float *sums, int64_t rows, int heads, float *dg, cudaStream_t stream) {
    dla_sum_decay_kernel<<<heads, kThreads, 0, stream>>>(sums, rows, heads, dg);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace dla

size_t dla_simt_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k, int32_t d_v, bool bwd) {
    return dla::space(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v, bwd).floats * 4;
}

cudaError_t launch_dla_simt(const DlaArgs &p, bool bwd, cudaStream_t stream) {
    using namespace dla;
    const int walks = bwd ? 2 : 1;
    if (p.n_tok > 0) {
        const dim3 grid((unsigned)n_slots(p.n_tok, p.n_seq), p.n_heads, walks * ((p.d_k + kDkBlock - 1) / kDkBlock));
        dla_simt_add_kernel<<<grid, kThreads, 0, stream>>>(p, bwd);
        count_launches(1);
    }
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && p.n_seq > 0) {
        const dim3 grid((unsigned)p.n_seq * p.n_heads, (p.d_k * p.d_v + kThreads - 1) / kThreads, walks);
        e = gdr::launch_dependent(dla_simt_walk_kernel, grid, kThreads, 0, stream, p, bwd);
    }
    if (e == cudaSuccess && p.n_tok > 0) {
        if (p.d_k <= 64) e = p.d_v <= 64 ? results<4, 4>(p, bwd, stream) : results<4, 8>(p, bwd, stream);
        else e = p.d_v <= 64 ? results<8, 4>(p, bwd, stream) : results<8, 8>(p, bwd, stream);
        if (e == cudaSuccess && bwd && p.n_heads > p.n_k_heads) {
            const int64_t n = p.n_tok * p.n_k_heads * p.d_k;
            e = gdr::launch_dependent(dla_simt_shared_heads_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads), 2), kThreads, 0, stream, p);
        }
    }
    if (e == cudaSuccess && bwd && p.dg && p.g_stride == 0) {
        const bool any = p.n_tok > 0;
        const float *sums = any ? static_cast<const float *>(p.workspace) +
                                      space(p.n_tok, p.n_seq, p.n_heads, p.n_k_heads, p.d_k, p.d_v, true).sums : nullptr;
        e = launch_dla_sum_decay(sums, any ? n_slots(p.n_tok, p.n_seq) : 0, p.n_heads, p.dg, stream);
    }
    return e;
}

}  // namespace kda
