// kda_dla_simt.cu -- linear attention with one decay per head without tensor cores, forward and
// backward; the formulas are in kda_dla.h.
//
// Chunks of 64 tokens. One launch walks over the chunks of every sequence and leaves the state at
// each chunk's start (and, backward, the gradient of each chunk's end state) in the workspace; a
// second one forms every chunk's results, all chunks side by side. Products are fp32 FMAs on tiles in
// shared memory, a thread holding 4 rows x 8 columns of a 64 x 128 result: per step of the
// contraction 32 FMAs for 9 reads, so that the FMA pipe bounds a chunk.
#include <cuda_bf16.h>

#include "kda_dla.h"

namespace kda {
namespace dla {
namespace {

constexpr int C = 64, kThreads = 256;
constexpr int LD = 132;  // floats between rows of a tile: rows 4 banks apart
constexpr int LW = 68;   // of the 64 x 64 pair weights
constexpr int kDkBlock = 32;

__device__ __forceinline__ float get(const float *p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

struct Gates {
    float2 G[C];     // sums of g log2(e) up to and with each token
    float gam[C], del[C], whole;
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
    if (lane == 0) out->whole = exp2_of(total);
}

// rows x cols of src into a tile of 64 x 128, zeros beyond
template <typename T>
__device__ __forceinline__ void load_tile(float *dst, const T *src, int64_t stride, int rows, int cols) {
    for (int i = threadIdx.x; i < C * 128; i += kThreads) {
        const int r = i >> 7, c = i & 127;
        dst[r * LD + c] = r < rows && c < cols ? get(src + r * stride + c) : 0.f;
    }
}

// A thread's part of a product: rows 4 tr + i, columns tc + 16 j
__device__ __forceinline__ int tr() { return threadIdx.x >> 4; }
__device__ __forceinline__ int tc() { return threadIdx.x & 15; }
// acc += A B, A (64 x n) and B (n x 16 NJ) by rows; n a multiple of 4
template <int NJ>
__device__ __forceinline__ void mm_nn(float (*acc)[NJ], const float *A, int lda, const float *B, int n) {
    const float *a = A + 4 * tr() * lda, *b = B + tc();
    for (int k = 0; k < n; k += 4) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(a + i * lda + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const float y = b[(k + kk) * LD + 16 * j];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = fmaf((&x[i].x)[kk], y, acc[i][j]);
            }
    }
}
// acc += A B^T, B (16 NJ x n) by rows
template <int NJ>
__device__ __forceinline__ void mm_nt(float (*acc)[NJ], const float *A, const float *B, int n) {
    const float *a = A + 4 * tr() * LD, *b = B + tc() * LD;
    for (int k = 0; k < n; k += 4) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(a + i * LD + k);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float4 y = *reinterpret_cast<const float4 *>(b + 16 * j * LD + k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i][j] = fmaf(x[i].w, y.w, fmaf(x[i].z, y.z, fmaf(x[i].y, y.y, fmaf(x[i].x, y.x, acc[i][j]))));
        }
    }
}
// acc += A^T B, A (64 x 64, rows LW apart) and B (64 x 16 NJ) by rows, over the rows from k0
template <int NJ>
__device__ __forceinline__ void mm_tn(float (*acc)[NJ], const float *A, const float *B, int n) {
    const float *a = A + 4 * tr(), *b = B + tc();
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(a + k * LW);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float y = b[k * LD + 16 * j];
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
// over the 16 threads that share rows
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ size_t state_size(const DlaArgs &p) { return (size_t)p.d_k * p.d_v; }
// the state at a chunk's start, then (backward) the gradients of the chunks' end states
__device__ __forceinline__ float *chunk_state(const DlaArgs &p, int64_t slot, int head, bool reverse) {
    float *ws = static_cast<float *>(p.workspace);
    return ws + ((reverse ? n_slots(p.n_tok, p.n_seq) : 0) + slot) * p.n_heads * state_size(p) + head * state_size(p);
}

// ---------------------------------------------------------------- states
// One CTA per (sequence, head, 32 key channels), backward also per direction: 32 x d_v of the
// state in registers, 4 x 4 a thread; the next chunk's rows are fetched while this one's are added.
template <typename T>
__global__ void __launch_bounds__(kThreads) dla_simt_states_kernel(const DlaArgs p, bool bwd) {
    __shared__ __align__(16) float ks[C][kDkBlock], vs[C][128];
    __shared__ Gates gate;
    const int n_blk = (p.d_k + kDkBlock - 1) / kDkBlock;
    unsigned b = blockIdx.x;
    const int blk = b % n_blk;
    b /= n_blk;
    const int head = b % p.n_heads;
    b /= p.n_heads;
    const int seq = b % p.n_seq;
    const bool rev = bwd && b / p.n_seq == 0;  // the reverse walks first
    const int kh = head / (p.n_heads / p.n_k_heads), i0 = blk * kDkBlock, tid = threadIdx.x;
    const int64_t start = p.cu_seqlens[seq], len = p.cu_seqlens[seq + 1] - start;
    const int nc = (int)((len + C - 1) / C);
    const int64_t slot0 = slot_base(p.cu_seqlens, seq);
    const int ti = (tid >> 5) * 4, tj = (tid & 31) * 4;
    const float *from = rev ? p.dh_final : p.h0;
    const int64_t at = ((int64_t)seq * p.n_heads + head) * state_size(p);
    auto in = [&](int i, int j) { return i0 + ti + i < p.d_k && tj + j < p.d_v; };
    auto pos = [&](int i, int j) { return (int64_t)(i0 + ti + i) * p.d_v + tj + j; };
    float S[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[i][j] = from && in(i, j) ? from[at + pos(i, j)] : 0.f;
    const T *key = static_cast<const T *>(rev ? p.q : p.k) + (int64_t)kh * p.d_k + i0;
    const int64_t key_stride = rev ? p.q_stride : p.k_stride, val_stride = rev ? (int64_t)p.n_heads * p.d_v : p.v_stride;
    const T *val = static_cast<const T *>(rev ? p.dout : p.v) + (int64_t)head * p.d_v;
    float kx[C * kDkBlock / kThreads], vx[C * 128 / kThreads];
    auto fetch = [&](int c) {
        const int64_t t0 = start + (int64_t)c * C;
        const int left = (int)min((int64_t)C, len - (int64_t)c * C);
#pragma unroll
        for (int x = 0; x < C * kDkBlock / kThreads; ++x) {
            const int r = (tid + x * kThreads) / kDkBlock, i = tid % kDkBlock;
            kx[x] = r < left && i0 + i < p.d_k ? get(key + (t0 + r) * key_stride + i) : 0.f;
        }
#pragma unroll
        for (int x = 0; x < C * 128 / kThreads; ++x) {
            const int r = (tid + x * kThreads) / 128, j = tid % 128;
            vx[x] = r < left && j < p.d_v ? get(val + (t0 + r) * val_stride + j) : 0.f;
        }
    };
    if (nc > 0) fetch(rev ? nc - 1 : 0);
    for (int n = 0; n < nc; ++n) {
        const int c = rev ? nc - 1 - n : n;
        float *keep = chunk_state(p, slot0 + c, head, rev);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in(i, j)) keep[pos(i, j)] = S[i][j];
        __syncthreads();  // the last chunk's rows are read
        if (tid < 32) {
            const int64_t t0 = start + (int64_t)c * C;
            chunk_gates(p, {seq, (int)min((int64_t)C, len - (int64_t)c * C), t0}, head, &gate);
        }
#pragma unroll
        for (int x = 0; x < C * kDkBlock / kThreads; ++x) ks[(tid + x * kThreads) / kDkBlock][tid % kDkBlock] = kx[x];
        __syncthreads();
        // the decay goes to the values: one factor a row
#pragma unroll
        for (int x = 0; x < C * 128 / kThreads; ++x) {
            const int r = (tid + x * kThreads) / 128;
            vs[r][tid % 128] = vx[x] * (rev ? p.scale * gate.gam[r] : gate.del[r]);
        }
        __syncthreads();
        if (n + 1 < nc) fetch(rev ? c - 1 : c + 1);
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
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[i][j] = fmaf(gate.whole, S[i][j], add[i][j]);
    }
    float *to = rev ? p.dh0 : p.h_final;
    if (!to) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (in(i, j)) to[at + pos(i, j)] = S[i][j];
}

// ---------------------------------------------------------------- output
struct OutSmem {
    float q[C * LD], k[C * LD], v[C * LD], s[128 * LD], w[C * LW];
    Gates gate;
};
__device__ __forceinline__ void load_state(float *dst, const float *src, int d_k, int d_v) {
    for (int i = threadIdx.x; i < 128 * 128; i += kThreads) {
        const int r = i >> 7, c = i & 127;
        dst[r * LD + c] = r < d_k && c < d_v ? src[(int64_t)r * d_v + c] : 0.f;
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

template <typename T>
__global__ void __launch_bounds__(kThreads) dla_simt_out_kernel(const DlaArgs p) {
    extern __shared__ __align__(16) char smem_raw[];
    OutSmem &s = *reinterpret_cast<OutSmem *>(smem_raw);
    const int64_t slot = blockIdx.x;
    const Chunk ch = find_chunk(p.cu_seqlens, p.n_seq, slot);
    if (ch.len == 0) return;
    const int head = blockIdx.y, kh = head / (p.n_heads / p.n_k_heads);
    load_tile(s.q, static_cast<const T *>(p.q) + ch.t0 * p.q_stride + (int64_t)kh * p.d_k, p.q_stride, ch.len, p.d_k);
    load_tile(s.k, static_cast<const T *>(p.k) + ch.t0 * p.k_stride + (int64_t)kh * p.d_k, p.k_stride, ch.len, p.d_k);
    load_tile(s.v, static_cast<const T *>(p.v) + ch.t0 * p.v_stride + (int64_t)head * p.d_v, p.v_stride, ch.len, p.d_v);
    load_state(s.s, chunk_state(p, slot, head, false), p.d_k, p.d_v);
    if (threadIdx.x < 32) chunk_gates(p, ch, head, &s.gate);
    __syncthreads();
    const int dk4 = (p.d_k + 3) & ~3;
    float qk[4][4], o[4][8];
    clear<4>(qk);
    mm_nt<4>(qk, s.q, s.k, dk4);
    weights(s.w, qk, s.gate, p.scale);
    clear<8>(o);
    mm_nn<8>(o, s.q, LD, s.s, dk4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f = p.scale * s.gate.gam[4 * tr() + i];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[i][j] *= f;
    }
    __syncthreads();
    mm_nn<8>(o, s.w, LW, s.v, C);
    T *out = static_cast<T *>(p.out) + (ch.t0 * p.n_heads + head) * p.d_v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * tr() + i;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = tc() + 16 * j;
            if (r < ch.len && c < p.d_v) put(out + (int64_t)r * p.n_heads * p.d_v + c, o[i][j]);
        }
    }
}

// ---------------------------------------------------------------- gradients
// One CTA per (chunk, key head): it walks over the value heads that share the key head and adds
// their dQ and dK in registers.
struct GradSmem {
    float q[C * LD], k[C * LD], v[C * LD], d[C * LD], s[128 * LD], w[C * LW];
    Gates gate;
    float a[C], b[C], row[C], col[8][C], ss[8];
};

template <typename T>
__global__ void __launch_bounds__(kThreads) dla_simt_grad_kernel(const DlaArgs p, float *sums) {
    extern __shared__ __align__(16) char smem_raw[];
    GradSmem &s = *reinterpret_cast<GradSmem *>(smem_raw);
    const int64_t slot = blockIdx.x;
    const Chunk ch = find_chunk(p.cu_seqlens, p.n_seq, slot);
    const int kh = blockIdx.y, group = p.n_heads / p.n_k_heads, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (ch.len == 0) {
        if (sums)
            for (int hh = tid; hh < group; hh += kThreads) sums[slot * p.n_heads + kh * group + hh] = 0.f;
        return;
    }
    load_tile(s.q, static_cast<const T *>(p.q) + ch.t0 * p.q_stride + (int64_t)kh * p.d_k, p.q_stride, ch.len, p.d_k);
    load_tile(s.k, static_cast<const T *>(p.k) + ch.t0 * p.k_stride + (int64_t)kh * p.d_k, p.k_stride, ch.len, p.d_k);
    const int dk4 = (p.d_k + 3) & ~3, dv4 = (p.d_v + 3) & ~3;
    const int64_t row = (int64_t)p.n_heads * p.d_v;
    float dq[4][8], dk[4][8];
    clear<8>(dq);
    clear<8>(dk);
    for (int hh = 0; hh < group; ++hh) {
        const int head = kh * group + hh;
        __syncthreads();
        load_tile(s.v, static_cast<const T *>(p.v) + ch.t0 * p.v_stride + (int64_t)head * p.d_v, p.v_stride, ch.len, p.d_v);
        load_tile(s.d, static_cast<const T *>(p.dout) + ch.t0 * row + (int64_t)head * p.d_v, row, ch.len, p.d_v);
        load_state(s.s, chunk_state(p, slot, head, false), p.d_k, p.d_v);
        if (warp == 0) chunk_gates(p, ch, head, &s.gate);
        __syncthreads();
        float x[4][8], qk[4][4], ov[4][4];
        clear<8>(x);
        mm_nt<8>(x, s.d, s.s, dv4);  // dO S0^T
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * tr() + i;
            const float f = p.scale * s.gate.gam[r];
            float a = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a = fmaf(s.q[r * LD + tc() + 16 * j], x[i][j], a);
                dq[i][j] = fmaf(f, x[i][j], dq[i][j]);
            }
            a = row_sum(a);
            if (tc() == 0) s.a[r] = f * a;
        }
        clear<4>(qk);
        clear<4>(ov);
        mm_nt<4>(qk, s.q, s.k, dk4);
        mm_nt<4>(ov, s.d, s.v, dv4);
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
        mm_nn<8>(dq, s.w, LW, s.k, C);
        mm_tn<8>(dk, s.w, s.q, C);
        __syncthreads();
        const float *end = chunk_state(p, slot, head, true);
        float ss = 0.f;
        for (int i = tid; i < 128 * 128; i += kThreads) {
            const int r = i >> 7, c = i & 127;
            const float y = r < p.d_k && c < p.d_v ? end[(int64_t)r * p.d_v + c] : 0.f;
            ss = fmaf(s.s[r * LD + c], y, ss);
            s.s[r * LD + c] = y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) s.ss[warp] = ss;
        weights(s.w, qk, s.gate, p.scale);
        __syncthreads();
        clear<8>(x);
        mm_nt<8>(x, s.v, s.s, dv4);  // V dS1^T
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * tr() + i;
            const float f = s.gate.del[r];
            float b = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                b = fmaf(s.k[r * LD + tc() + 16 * j], x[i][j], b);
                dk[i][j] = fmaf(f, x[i][j], dk[i][j]);
            }
            b = row_sum(b);
            if (tc() == 0) s.b[r] = f * b;
        }
        clear<8>(x);
        mm_nn<8>(x, s.k, LD, s.s, dk4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = s.gate.del[4 * tr() + i];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] *= f;
        }
        mm_tn<8>(x, s.w, s.d, C);
        T *dv = static_cast<T *>(p.dv) + ch.t0 * row + (int64_t)head * p.d_v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * tr() + i;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = tc() + 16 * j;
                if (r < ch.len && c < p.d_v) put(dv + r * row + c, x[i][j]);
            }
        }
        if (!p.dg) continue;
        __syncthreads();
        if (warp == 0) {  // two tokens a lane, running sums over the chunk
            float whole = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) whole += s.ss[i];
            whole *= s.gate.whole;
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
    T *gq = static_cast<T *>(p.dq) + (ch.t0 * p.n_k_heads + kh) * p.d_k;
    T *gk = static_cast<T *>(p.dk) + (ch.t0 * p.n_k_heads + kh) * p.d_k;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * tr() + i;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = tc() + 16 * j;
            if (r < ch.len && c < p.d_k) {
                put(gq + (int64_t)r * p.n_k_heads * p.d_k + c, dq[i][j]);
                put(gk + (int64_t)r * p.n_k_heads * p.d_k + c, dk[i][j]);
            }
        }
    }
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

}  // namespace

cudaError_t launch_dla_sum_decay(const float *sums, int64_t rows, int heads, float *dg, cudaStream_t stream) {
    dla_sum_decay_kernel<<<heads, kThreads, 0, stream>>>(sums, rows, heads, dg);
    count_launches(1);
    return cudaGetLastError();
}

namespace {

template <typename T>
cudaError_t run(const DlaArgs &p, bool bwd, cudaStream_t stream) {
    const int64_t slots = n_slots(p.n_tok, p.n_seq);
    const unsigned blocks = (unsigned)((p.d_k + kDkBlock - 1) / kDkBlock) * p.n_heads * p.n_seq * (bwd ? 2 : 1);
    if (blocks > 0) {
        dla_simt_states_kernel<T><<<blocks, kThreads, 0, stream>>>(p, bwd);
        count_launches(1);
    }
    if (p.n_tok > 0) {
        cudaError_t e;
        if (!bwd) {
            e = allow_smem(reinterpret_cast<const void *>(dla_simt_out_kernel<T>), sizeof(OutSmem));
            if (e != cudaSuccess) return e;
            dla_simt_out_kernel<T><<<dim3((unsigned)slots, p.n_heads), kThreads, sizeof(OutSmem), stream>>>(p);
        } else {
            e = allow_smem(reinterpret_cast<const void *>(dla_simt_grad_kernel<T>), sizeof(GradSmem));
            if (e != cudaSuccess) return e;
            float *sums = p.dg && p.g_stride == 0
                              ? static_cast<float *>(p.workspace) + 2 * slots * p.n_heads * p.d_k * p.d_v
                              : nullptr;
            dla_simt_grad_kernel<T><<<dim3((unsigned)slots, p.n_k_heads), kThreads, sizeof(GradSmem), stream>>>(p, sums);
            if (sums) {
                e = launch_dla_sum_decay(sums, slots, p.n_heads, p.dg, stream);
                if (e != cudaSuccess) return e;
            }
        }
        count_launches(1);
    } else if (bwd && p.dg && p.g_stride == 0) {
        return launch_dla_sum_decay(nullptr, 0, p.n_heads, p.dg, stream);
    }
    return cudaGetLastError();
}

}  // namespace
}  // namespace dla

size_t dla_simt_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t d_k, int32_t d_v, bool bwd) {
    const size_t states = (size_t)gdr::n_slots(n_tok, n_seq) * n_heads;
    return (bwd ? 2 * states * d_k * d_v + states : states * d_k * d_v) * 4;  // bwd: and a chunk's sum of dg
}

cudaError_t launch_dla_simt(const DlaArgs &p, bool bwd, cudaStream_t stream) {
    return p.bf16 ? dla::run<__nv_bfloat16>(p, bwd, stream) : dla::run<float>(p, bwd, stream);
}

}  // namespace kda
