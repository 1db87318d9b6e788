// kda_gdr_fwd.cu -- chunked forward of the gated delta rule with one decay per head.
//
// Per sequence and value head, with a_t = exp(g_t):
//   S_t = a_t S_{t-1} + beta_t k_t (v_t - a_t S_{t-1}^T k_t)^T,   o_t = d_k^-1/2 S_t^T q_t.
// Over a chunk of 64 tokens with start state S0, D_rj = sum of g over (j, r],
// gamma_r = exp(sum of g up to r), delta_r = exp(sum of g past r), Gamma = gamma of the last:
//   A = strict_lower(beta_r e^D_rj k_r.k_j),  X = (I + A)^-1,  P = lower(e^D_rj q_r.k_j)
//   Z = V - gamma K S0,   U = X (beta Z),   O = d_k^-1/2 (gamma Q S0 + P U)
//   S1 = Gamma S0 + (delta K)^T U
// Unlike the per-channel decay, the scalar one leaves K and Q as they are and only scales
// rows, columns and pairs: no exponent above zero is formed, the decay is unbounded below.
//
// Two kernels. gdr_terms: X, P and the gates of every chunk, all chunks side by side. gdr_chain:
// the chunks of a sequence in order. A pair of warps owns 16 value channels and keeps their
// state transposed (16 x d_k) in registers for the whole sequence, each warp one half of d_k in
// fp32 and both all of it as bf16 planes. An fp32 accumulator tile of mma.sync lies in registers
// as the A operand (and as the B operand of the transposed product) of the next one, so
// S^T -> Y^T -> Z^T -> U^T -> S^T passes through shared memory only where the two warps trade
// halves. That serial path is what bounds the pass: a tcgen05 form pays commit, tensor-memory
// read, convert, store and fence at each of its hand-offs, and a chunk has four.
//
// bf16, d_k = d_v = 128: 64K tokens of 16 key and 32 value heads in one sequence take 2.43 ms, 0.42
// of it the terms and 1.98 the chains (1024 steps of 64 tokens); 20K tokens of 16 value heads in
// 12 sequences 0.39 ms. Both are far from the bytes they move (0.24 and 0.05 ms).
#include <cmath>

#include "kda_gdr_chain.h"

namespace kda {
namespace gdr {
namespace {

constexpr int kTermThreads = 256;
constexpr int kARow = 68;  // floats of a row of A in shared memory

template <int NI, int DKP>
struct TermsSmem {
    static constexpr int kPlane = C * DKP * 2;
    static constexpr int K = 0, Q = K + NI * kPlane;
    static constexpr int kKept = 24 * kTermThreads * 4;  // the products K K^T and Q K^T, over K and Q
    static constexpr int A = 2 * NI * kPlane > kKept ? 2 * NI * kPlane : kKept;
    static constexpr int Vec = A + 2 * C * kARow * 4;           // per head: G as float2, beta
    static constexpr int kBytes = Vec + 2 * 3 * C * 4;
};

constexpr float kLog2e = 1.44269502f, kLog2eLo = 1.92596299e-8f;  // log2(e) in two floats
// 2^(hi + lo), lo far below hi
__device__ __forceinline__ float exp2_of(float hi, float lo) {
    const float e = ex2(hi);
    return fmaf(e * 0.693147181f, lo, e);
}

// ---- the inverse of I + A, a head at a time by two warps, in place over A (fp32, rows kARow
// apart; strictly lower entries valid). 16 x 16 diagonal blocks by forward substitution, a
// column per thread; then [[X0, 0], [-X1 A10 X0, X1]] for pairs of 16-blocks and for the pair
// of 32-blocks, products of as many bf16 planes as X is kept in. M^T = X0^T A10^T is formed first: its
// accumulators are the B operand of X1 M, so M stays in registers.
template <int NS, int R>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (*w)[R], int i) {
    uint32_t s[NS];
    split2<NS>(x, y, s);
#pragma unroll
    for (int q = 0; q < NS; ++q) w[q][i] = s[q];
}
// D (16 x 8) += A B over planes i + j < NS
template <int NS>
__device__ __forceinline__ void mma_planes(float *d, const uint32_t (*a)[4], const uint32_t (*b)[2]) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int j = 0; i + j < NS; ++j) ptx::mma16816(d, a[i], b[j][0], b[j][1]);
}
__device__ __forceinline__ void diagonal_column(float *A, int b, int c, bool on) {
    const float *D = A + (16 * b) * kARow + 16 * b;
    float x[16];
    if (on)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        float s0 = r == c ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < r; ++k) {
            if (k & 1) s1 = fmaf(-D[r * kARow + k], x[k], s1);
            else s0 = fmaf(-D[r * kARow + k], x[k], s0);
        }
        x[r] = s0 + s1;
    }
    __syncthreads();
    if (on)
#pragma unroll
    for (int r = 0; r < 16; ++r) A[(16 * b + r) * kARow + 16 * b + c] = x[r];
}
// X block of size N at rows r0, columns c0 (its diagonal blocks at c0 and r0 done), columns
// n0 .. n0 + 15 of it; reads A10 first, writes after the barrier
template <int N, int NS>
__device__ __forceinline__ void join_blocks(float *A, int r0, int c0, int n0, bool on) {
    const int lane = threadIdx.x & 31, gr = lane >> 2, tq = lane & 3;
    float x[N / 16][2][4];
    if (on) {
        float m[N / 8][4];  // M^T: rows n0 .., columns the block's rows
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) m[i][j] = 0.f;
#pragma unroll
        for (int k = 0; k < N; k += 16) {
            uint32_t a[NS][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // X0^T[n][k] = X0[k][n]
                const int n = n0 + gr + (i & 1) * 8, kk = k + tq * 2 + (i >> 1) * 8;
                split_pair<NS>(A[(c0 + kk) * kARow + c0 + n], A[(c0 + kk + 1) * kARow + c0 + n], a, i);
            }
#pragma unroll
            for (int t = 0; t < N / 8; ++t) {
                uint32_t b[NS][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {  // A10[row][k]
                    const float2 v = *reinterpret_cast<const float2 *>(A + (r0 + t * 8 + gr) * kARow + c0 + k + tq * 2 + i * 8);
                    split_pair<NS>(v.x, v.y, b, i);
                }
                mma_planes<NS>(m[t], a, b);
            }
        }
#pragma unroll
        for (int i = 0; i < N / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][0][j] = x[i][1][j] = 0.f;
#pragma unroll
        for (int k = 0; k < N; k += 16) {
            uint32_t b0[NS][2], b1[NS][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float *t = m[k / 8 + i];
                split_pair<NS>(t[0], t[1], b0, i);
                split_pair<NS>(t[2], t[3], b1, i);
            }
#pragma unroll
            for (int mt = k / 16; mt < N / 16; ++mt) {  // X1 is lower triangular
                uint32_t a[NS][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = *reinterpret_cast<const float2 *>(A + (r0 + mt * 16 + gr + (i & 1) * 8) * kARow +
                                                                       r0 + k + tq * 2 + (i >> 1) * 8);
                    split_pair<NS>(v.x, v.y, a, i);
                }
                mma_planes<NS>(x[mt][0], a, b0);
                mma_planes<NS>(x[mt][1], a, b1);
            }
        }
    }
    __syncthreads();
    if (on)
#pragma unroll
        for (int mt = 0; mt < N / 16; ++mt)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2 *>(A + (r0 + mt * 16 + gr + 8 * h) * kARow + c0 + n0 + n * 8 + tq * 2) =
                        make_float2(-x[mt][n][2 * h], -x[mt][n][2 * h + 1]);
    __syncthreads();
}

// The ten 16 x 16 blocks on and below the diagonal, shared out over four warps: at most three
// each. w 0: (3,0) (3,1) (0,0)   1: (3,2) (1,0) (1,1)   2: (3,3) (2,0)   3: (2,1) (2,2)
__device__ __forceinline__ void block_of(int w, int s, int &I, int &J) {
    const uint32_t t = (w & 2 ? (w & 1 ? 0x2221u : 0x2033u) : (w & 1 ? 0x111032u : 0x003130u)) >> (8 * s);
    I = (t >> 4) & 15;
    J = t & 15;
}

// One CTA per (chunk, key head): the products K K^T and Q K^T once, then the value heads that share
// them, two at a time. The inverse is the one serial part; three CTAs an SM cover it and the
// kernel is bound by instruction issue (0.6 of the slots at 64K tokens of 16 key and 32 value
// heads, 0.42 ms; two CTAs an SM with the products in registers, P out in one plane: 0.49 ms, three then 0.41).
template <typename T, int DKP, int NS>
__global__ void __launch_bounds__(kTermThreads, InputPlanes<T>::N == 1 ? 3 : 1)
    gdr_terms_kernel(const GdrArgs p, const Images im, int values, float scale, bool vec) {
    constexpr int NI = InputPlanes<T>::N;
    using L = TermsSmem<NI, DKP>;
    extern __shared__ __align__(1024) char smem[];
    const uint32_t base = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tq = lane & 3;
    let_next_kernel_start();
    const int64_t slot = blockIdx.x;
    const Chunk ch = find_chunk(p.cu_seqlens, p.n_seq, slot);
    if (ch.len == 0) return;
    const int hk = p.n_k_heads, hv = p.n_heads, kh = blockIdx.y, group = hv / hk;
    char *ws = static_cast<char *>(p.workspace);
    float *A = reinterpret_cast<float *>(smem + L::A);
    float *vec_s = reinterpret_cast<float *>(smem + L::Vec);

    // The gates' inputs of the heads h0 and h0 + 1, a warp each, ahead of their use.
    float gx[2], bx[2];
    auto fetch_gates = [&](int h0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = lane * 2 + i;
            gx[i] = bx[i] = 0.f;
            if (warp < min(2, group - h0) && r < ch.len) {
                const int64_t at = (ch.t0 + r) * hv + kh * group + h0 + warp;
                gx[i] = p.g[at];
                bx[i] = p.beta[at];
            }
        }
    };
    fetch_gates(0);
    load_key_tile<T, DKP>(base + L::K, static_cast<const T *>(p.k) + ch.t0 * p.k_stride + (int64_t)kh * p.d_k,
                          p.k_stride, ch.len, p.d_k, vec, tid, kTermThreads);
    load_key_tile<T, DKP>(base + L::Q, static_cast<const T *>(p.q) + ch.t0 * p.q_stride + (int64_t)kh * p.d_k,
                          p.q_stride, ch.len, p.d_k, vec, tid, kTermThreads);
    ptx::cp_async_commit();

    // The gates of the heads h0 and h0 + 1, a warp each: running sums of g log2(e) in two floats,
    // so that differences of neighbours stay exact.
    auto gates = [&](int h0) {
        if (warp >= min(2, group - h0)) return;
        const int head = kh * group + h0 + warp;
        Two s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // below -200 (and at -inf) the decay is 0 in fp32 all the same; a finite floor keeps
            // differences of the sums free of inf - inf
            const float x = gx[i] < kGFloor ? kGFloor : gx[i];
            s[i].hi = x * kLog2e;
            s[i].lo = fmaf(x, kLog2e, -s[i].hi) + x * kLog2eLo;
        }
        s[1] = add(s[0], s[1]);
        Two run = s[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Two y = {__shfl_up_sync(0xffffffffu, run.hi, o), __shfl_up_sync(0xffffffffu, run.lo, o)};
            if (lane >= o) run = add(y, run);
        }
        Two before = {__shfl_up_sync(0xffffffffu, run.hi, 1), __shfl_up_sync(0xffffffffu, run.lo, 1)};
        if (lane == 0) before = {0.f, 0.f};
        const Two total = {__shfl_sync(0xffffffffu, run.hi, 31), __shfl_sync(0xffffffffu, run.lo, 31)};
        float *out = reinterpret_cast<float *>(ws + (slot * hv + head) * terms_bytes(NS) + 2 * NS * kTri);
        float2 *G2 = reinterpret_cast<float2 *>(vec_s + warp * 3 * C);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = lane * 2 + i;
            const Two G = i ? run : add(before, s[0]);
            G2[r] = make_float2(G.hi, G.lo);
            vec_s[warp * 3 * C + 2 * C + r] = bx[i];
            out[r] = exp2_of(G.hi, G.lo);
            out[C + r] = ex2((total.hi - G.hi) + (total.lo - G.lo));
            out[2 * C + r] = bx[i];
            out[3 * C + r] = exp2_of(total.hi, total.lo);
            reinterpret_cast<float2 *>(out + 4 * C)[r] = make_float2(G.hi, G.lo);
        }
    };
    gates(0);  // while the tiles arrive
    cp_async_wait<0>();
    __syncthreads();

    if (im.has(ch.t0, ch.len, p.n_tok)) {
        const size_t rec = Images::record(NI, DKP, p.d_v, hk, hv, values), kb = Images::key_bytes(NI, DKP);
        const size_t vb = Images::value_bytes(NI, p.d_v);
        char *img = ws + im.offset + (im.all ? slot : (int64_t)ch.seq) * rec;
        for (int i = tid; i < NI * L::kPlane / 16; i += kTermThreads) {
            reinterpret_cast<uint4 *>(img + kh * kb)[i] = reinterpret_cast<const uint4 *>(smem + L::Q)[i];
            reinterpret_cast<uint4 *>(img + (hk + kh) * kb)[i] = reinterpret_cast<const uint4 *>(smem + L::K)[i];
        }
        write_value_images<T>(img + 2 * hk * kb + kh * group * vb, vb,
                              static_cast<const T *>(p.v) + ch.t0 * p.v_stride + (int64_t)kh * group * p.d_v,
                              p.v_stride, group, ch.len, p.d_v, tid, kTermThreads);
        if (values == 2)
            write_value_images<T>(img + 2 * hk * kb + (hv + kh * group) * vb, vb,
                                  static_cast<const T *>(p.dout) + (ch.t0 * hv + kh * group) * p.d_v,
                                  (int64_t)hv * p.d_v, group, ch.len, p.d_v, tid, kTermThreads);
    }

    // K K^T (warps 0..3) and Q K^T (warps 4..7), the blocks of block_of()
    const int wr = warp & 3, nb = wr < 2 ? 3 : 2;
    const bool keys = warp < 4;
    int I[3], J[3];
#pragma unroll
    for (int s = 0; s < 3; ++s) block_of(wr, s < nb ? s : 0, I[s], J[s]);
    float kk[3][2][4];
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) kk[s][0][i] = kk[s][1][i] = 0.f;
#pragma unroll 2
    for (int c = 0; c < DKP; c += 16)
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            if (s >= nb) break;
            uint32_t a[NI][4];
#pragma unroll
            for (int q = 0; q < NI; ++q) key_a(base + (keys ? L::K : L::Q) + q * L::kPlane, I[s] * 16, c, a[q]);
            uint32_t b[NI][4];
#pragma unroll
            for (int q = 0; q < NI; ++q) key_b(base + L::K + q * L::kPlane, J[s] * 16, c, b[q]);
            product<NI, NI, NI>(kk[s], a, b);
        }

    // kept by each thread for itself over K and Q: 24 registers fewer, which three CTAs an SM need
    __syncthreads();
    float *kept = reinterpret_cast<float *>(smem + L::K) + tid;
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) kept[(s * 8 + i) * kTermThreads] = kk[s][i >> 2][i & 3];

    for (int h0 = 0; h0 < group; h0 += 2) {
        const int nh = min(2, group - h0);
        if (h0) {
            __syncthreads();  // A and the gates of the pair before are done with
            gates(h0);
            __syncthreads();
        }
        fetch_gates(h0 + 2);
        // A (fp32, to shared memory; warps 0..3) and P (bf16 planes, to the workspace; warps 4..7)
        for (int hh = 0; hh < nh; ++hh) {
            const float2 *G2 = reinterpret_cast<const float2 *>(vec_s + hh * 3 * C);
            const float *B = vec_s + hh * 3 * C + 2 * C;
            float *Ah = A + hh * C * kARow;
            char *P = ws + (slot * hv + kh * group + h0 + hh) * terms_bytes(NS) + NS * kTri;
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                if (s >= nb) break;
                const int r0 = I[s] * 16 + gr;
                const float2 g0 = G2[r0], g1 = G2[r0 + 8];
                const float f0 = keys ? B[r0] : scale, f1 = keys ? B[r0 + 8] : scale;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int j = J[s] * 16 + n * 8 + tq * 2;
                    const float4 gj = *reinterpret_cast<const float4 *>(&G2[j]);
                    const float *k4 = kept + (s * 8 + n * 4) * kTermThreads;
                    float x[4];
                    x[0] = f0 * k4[0] * ex2((g0.x - gj.x) + (g0.y - gj.y));
                    x[1] = f0 * k4[kTermThreads] * ex2((g0.x - gj.z) + (g0.y - gj.w));
                    x[2] = f1 * k4[2 * kTermThreads] * ex2((g1.x - gj.x) + (g1.y - gj.y));
                    x[3] = f1 * k4[3 * kTermThreads] * ex2((g1.x - gj.z) + (g1.y - gj.w));
                    if (I[s] == J[s]) {  // A is strictly lower triangular, P lower
                        const int e = keys ? 0 : 1;
                        if (j >= r0 + e) x[0] = 0.f;
                        if (j + 1 >= r0 + e) x[1] = 0.f;
                        if (j >= r0 + 8 + e) x[2] = 0.f;
                        if (j + 1 >= r0 + 8 + e) x[3] = 0.f;
                    }
                    if (keys) {
                        *reinterpret_cast<float2 *>(Ah + r0 * kARow + j) = make_float2(x[0], x[1]);
                        *reinterpret_cast<float2 *>(Ah + (r0 + 8) * kARow + j) = make_float2(x[2], x[3]);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t w[NS];
                            split2<NS>(x[2 * h], x[2 * h + 1], w);
                            char *at = P + tri_block(I[s], J[s]) + tile_off<32>(gr + 8 * h, n * 8 + tq * 2);
#pragma unroll
                            for (int pl = 0; pl < NS; ++pl) *reinterpret_cast<uint32_t *>(at + pl * kTri) = w[pl];
                        }
                    }
                }
            }
            if (wr == 3 && !keys) {  // the block above the diagonal that join_blocks<32> reads
#pragma unroll
                for (int i = 0; i < 8; ++i) Ah[(lane >> 1) * kARow + 16 + (lane & 1) * 8 + i] = 0.f;
            }
        }
        __syncthreads();
        // X in place: warps 2 h, 2 h + 1 for head h (the other warps only keep the barriers)
        {
            const int hh = warp >> 1, w = warp & 1, t = tid & 63;
            const bool on = hh < nh;
            float *X = A + (on ? hh : 0) * C * kARow;
            diagonal_column(X, t >> 4, t & 15, on);
            __syncthreads();
            join_blocks<16, NS>(X, 32 * w + 16, 32 * w, 0, on);
            join_blocks<32, NS>(X, 32, 0, 16 * w, on);
        }
        for (int i = tid; i < nh * 320; i += kTermThreads) {  // X out, split into planes on the way
            const int hh = i / 320, k = i % 320, b = k >> 5, r = (k >> 1) & 15, c = (k & 1) * 8;
            const int bi = b >= 6 ? 3 : b >= 3 ? 2 : b >= 1 ? 1 : 0, bj = b - bi * (bi + 1) / 2;
            const float *src = A + hh * C * kARow + (bi * 16 + r) * kARow + bj * 16 + c;
            char *dst = ws + (slot * hv + kh * group + h0 + hh) * terms_bytes(NS) + b * 512 + tile_off<32>(r, c);
            const float4 u = *reinterpret_cast<const float4 *>(src), v = *reinterpret_cast<const float4 *>(src + 4);
            uint32_t w[4][NS];
            split2<NS>(u.x, u.y, w[0]);
            split2<NS>(u.z, u.w, w[1]);
            split2<NS>(v.x, v.y, w[2]);
            split2<NS>(v.z, v.w, w[3]);
#pragma unroll
            for (int q = 0; q < NS; ++q)
                *reinterpret_cast<uint4 *>(dst + q * kTri) = make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
        }
    }
}

template <typename T, int DKP, int NS>
__global__ void __launch_bounds__(kChainThreads)
    gdr_chain_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const GdrArgs p, const Images im, float scale,
                     bool wide_out) {
    chain<T, DKP, NS, Mode::kForward, 2>(tm_q, tm_k, tm_v, p, im, 1, blockIdx.x, scale, wide_out);
}

template <typename T, int DKP, int NS>
cudaError_t terms(const GdrArgs &p, const Images &im, int values, cudaStream_t stream) {
    constexpr int bytes = TermsSmem<InputPlanes<T>::N, DKP>::kBytes;
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(gdr_terms_kernel<T, DKP, NS>), bytes);
    if (e != cudaSuccess) return e;
    const bool vec = rows_vec<T>(p.q, p.q_stride, p.d_k) && rows_vec<T>(p.k, p.k_stride, p.d_k);
    const dim3 grid((unsigned)n_slots(p.n_tok, p.n_seq), p.n_k_heads);
    gdr_terms_kernel<T, DKP, NS><<<grid, kTermThreads, bytes, stream>>>(p, im, values, 1.f / std::sqrt((float)p.d_k), vec);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int DKP>
cudaError_t forward(const GdrArgs &p, cudaStream_t stream) {
    constexpr int NI = InputPlanes<T>::N, NS = NI == 1 ? 2 : 3;
    ChainMaps maps;
    const Images im{!maps.make<T>(p, false), scan_offset(p.n_tok, p.n_seq, p.n_heads, NS)};
    cudaError_t e = launch_gdr_terms(p, im, 1, NS, stream);
    if (e != cudaSuccess) return e;
    const bool wide = p.d_v % 2 == 0 && ((uintptr_t)p.out % (2 * sizeof(T))) == 0;
    return launch_dependent(gdr_chain_kernel<T, DKP, NS>, chain_blocks(p, 2), kChainThreads,
                            ChainSmem<NI, DKP, NS, Mode::kForward, 2>::kBytes, stream, maps.q, maps.k, maps.v, p, im,
                            1.f / std::sqrt((float)p.d_k), wide);
}

}  // namespace
}  // namespace gdr

size_t gdr_fwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k,
                               int32_t d_v, bool bf16) {
    return gdr::scan_offset(n_tok, n_seq, n_heads, bf16 ? 2 : 3) +
           (size_t)gdr::n_slots(n_tok, n_seq) *
               gdr::Images::record(bf16 ? 1 : 3, d_k <= 64 ? 64 : 128, d_v, n_k_heads, n_heads, 1);
}

cudaError_t launch_gdr_terms(const GdrArgs &p, gdr::Images im, int values, int ns, cudaStream_t stream) {
    using bf16 = __nv_bfloat16;
    if (p.n_tok == 0) return cudaSuccess;
    if (!p.bf16) return p.d_k <= 64 ? gdr::terms<float, 64, 3>(p, im, values, stream) : gdr::terms<float, 128, 3>(p, im, values, stream);
    if (ns == 3) return p.d_k <= 64 ? gdr::terms<bf16, 64, 3>(p, im, values, stream) : gdr::terms<bf16, 128, 3>(p, im, values, stream);
    return p.d_k <= 64 ? gdr::terms<bf16, 64, 2>(p, im, values, stream) : gdr::terms<bf16, 128, 2>(p, im, values, stream);
}

cudaError_t launch_gdr_fwd(const GdrArgs &p, cudaStream_t stream) {
    if (p.bf16) return p.d_k <= 64 ? gdr::forward<__nv_bfloat16, 64>(p, stream) : gdr::forward<__nv_bfloat16, 128>(p, stream);
    return p.d_k <= 64 ? gdr::forward<float, 64>(p, stream) : gdr::forward<float, 128>(p, stream);
}

cudaError_t read_gdr_fwd_flags(unsigned int *flags, bool reset, cudaStream_t stream) {
    return gdr::read_flags(flags, reset, stream);
}

}  // namespace kda
