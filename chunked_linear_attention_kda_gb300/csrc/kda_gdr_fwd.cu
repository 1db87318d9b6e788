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
// Two kernels. gdr_terms: X, P and the gates of every chunk, all chunks side by side.
// gdr_chain: the chunks of a sequence in order. A warp owns 16 value channels and keeps
// their state transposed (16 x d_k, fp32) in registers for the whole sequence. An fp32
// accumulator tile of mma.sync lies in registers as the A operand (and as the B operand of
// the transposed product) of the next one, so S^T -> Y^T -> Z^T -> U^T -> S^T never leaves
// the warp: no barrier and no shared-memory round trip sits on the serial path, which is
// what bounds this kernel (a tcgen05 form pays commit, tensor-memory read, convert, store
// and fence at each of these hand-offs).
#include <cmath>

#include "kda_gdr_chain.h"

namespace kda {
namespace gdr {
namespace {

constexpr int kTermThreads = 128;
constexpr int kARow = 68;  // floats of a row of A in shared memory

template <int NI, int DKP>
struct TermsSmem {
    static constexpr int NS = NI == 1 ? 2 : 3;
    static constexpr int kPlane = C * DKP * 2;
    static constexpr int K = 0, Q = K + NI * kPlane;
    static constexpr int kTileP = NS * kTile * 2;               // P of one head, over K or Q once they are used
    static constexpr int kHead = kTileP > NI * kPlane ? kTileP : NI * kPlane;
    static constexpr int A = 2 * kHead;
    static constexpr int Vec = A + 2 * C * kARow * 4;           // per head: Ghi, Glo, beta
    static constexpr int kBytes = Vec + 2 * 3 * C * 4;
};

// ---- the inverse of I + A, a head at a time by two warps, in place over A (fp32, rows kARow
// apart; strictly lower entries valid). 16 x 16 diagonal blocks by forward substitution, a
// column per thread; then [[X0, 0], [-X1 A10 X0, X1]] for pairs of 16-blocks and for the pair
// of 32-blocks, products of three bf16 planes (2^-24). M^T = X0^T A10^T is formed first: its
// accumulators are the B operand of X1 M, so M stays in registers.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (*w)[4], int i) {
    uint32_t s[3];
    split2<3>(x, y, s);
    w[0][i] = s[0]; w[1][i] = s[1]; w[2][i] = s[2];
}
// D (16 x 8) += A B over planes i + j < 3
__device__ __forceinline__ void mma3(float *d, const uint32_t (*a)[4], const uint32_t (*b)[2]) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; i + j < 3; ++j) ptx::mma16816(d, a[i], b[j][0], b[j][1]);
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
template <int N>
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
            uint32_t a[3][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // X0^T[n][k] = X0[k][n]
                const int n = n0 + gr + (i & 1) * 8, kk = k + tq * 2 + (i >> 1) * 8;
                split_pair(A[(c0 + kk) * kARow + c0 + n], A[(c0 + kk + 1) * kARow + c0 + n], a, i);
            }
#pragma unroll
            for (int t = 0; t < N / 8; ++t) {
                uint32_t b[3][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {  // A10[row][k]
                    const float2 v = *reinterpret_cast<const float2 *>(A + (r0 + t * 8 + gr) * kARow + c0 + k + tq * 2 + i * 8);
                    uint32_t s[3];
                    split2<3>(v.x, v.y, s);
                    b[0][i] = s[0]; b[1][i] = s[1]; b[2][i] = s[2];
                }
                mma3(m[t], a, b);
            }
        }
#pragma unroll
        for (int i = 0; i < N / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][0][j] = x[i][1][j] = 0.f;
#pragma unroll
        for (int k = 0; k < N; k += 16) {
            uint32_t b0[3][2], b1[3][2], s[3];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float *t = m[k / 8 + i];
                split2<3>(t[0], t[1], s);
                b0[0][i] = s[0]; b0[1][i] = s[1]; b0[2][i] = s[2];
                split2<3>(t[2], t[3], s);
                b1[0][i] = s[0]; b1[1][i] = s[1]; b1[2][i] = s[2];
            }
#pragma unroll
            for (int mt = k / 16; mt < N / 16; ++mt) {  // X1 is lower triangular
                uint32_t a[3][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = *reinterpret_cast<const float2 *>(A + (r0 + mt * 16 + gr + (i & 1) * 8) * kARow +
                                                                       r0 + k + tq * 2 + (i >> 1) * 8);
                    split_pair(v.x, v.y, a, i);
                }
                mma3(x[mt][0], a, b0);
                mma3(x[mt][1], a, b1);
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

template <typename T, int DKP>
__global__ void __launch_bounds__(kTermThreads)
    gdr_terms_kernel(const GdrArgs p, const Images im, int values, float scale, bool vec) {
    constexpr int NI = InputPlanes<T>::N, NS = NI == 1 ? 2 : 3;
    using L = TermsSmem<NI, DKP>;
    extern __shared__ __align__(1024) char smem[];
    const uint32_t base = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t slot = blockIdx.x;
    const Chunk ch = find_chunk(p.cu_seqlens, p.n_seq, slot);
    if (ch.len == 0) return;
    const int hk = p.n_k_heads, hv = p.n_heads, kh = blockIdx.y, group = hv / hk;
    char *ws = static_cast<char *>(p.workspace);

    load_key_tile<T, DKP>(base + L::K, static_cast<const T *>(p.k) + ch.t0 * p.k_stride + (int64_t)kh * p.d_k,
                          p.k_stride, ch.len, p.d_k, vec, tid, kTermThreads);
    load_key_tile<T, DKP>(base + L::Q, static_cast<const T *>(p.q) + ch.t0 * p.q_stride + (int64_t)kh * p.d_k,
                          p.q_stride, ch.len, p.d_k, vec, tid, kTermThreads);
    ptx::cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();

    if (im.all || ch.len < C) {
        const size_t rec = Images::record(NI, DKP, p.d_v, hk, hv, values), kb = Images::key_bytes(NI, DKP);
        const size_t vb = Images::value_bytes(NI, p.d_v);
        char *img = ws + im.offset + (im.all ? slot : (int64_t)ch.seq) * rec;
        for (int i = tid; i < NI * L::kPlane / 16; i += kTermThreads) {
            reinterpret_cast<uint4 *>(img + kh * kb)[i] = reinterpret_cast<const uint4 *>(smem + L::Q)[i];
            reinterpret_cast<uint4 *>(img + (hk + kh) * kb)[i] = reinterpret_cast<const uint4 *>(smem + L::K)[i];
        }
        for (int head = kh * group; head < (kh + 1) * group; ++head) {
            write_value_image<T>(img + 2 * hk * kb + head * vb,
                                 static_cast<const T *>(p.v) + ch.t0 * p.v_stride + (int64_t)head * p.d_v,
                                 p.v_stride, ch.len, p.d_v, tid, kTermThreads);
            if (values == 2)
                write_value_image<T>(img + 2 * hk * kb + (hv + head) * vb,
                                     static_cast<const T *>(p.dout) + (ch.t0 * hv + head) * p.d_v,
                                     (int64_t)hv * p.d_v, ch.len, p.d_v, tid, kTermThreads);
        }
    }

    // K K^T and Q K^T: warp w the rows 16 w .., columns up to its own
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) kk[n][i] = qk[n][i] = 0.f;
#pragma unroll 2
    for (int c = 0; c < DKP; c += 16) {
        uint32_t ak[NI][4], aq[NI][4];
#pragma unroll
        for (int q = 0; q < NI; ++q) {
            key_a(base + L::K + q * L::kPlane, warp * 16, c, ak[q]);
            key_a(base + L::Q + q * L::kPlane, warp * 16, c, aq[q]);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n > warp) break;
#pragma unroll
            for (int pb = 0; pb < NI; ++pb) {
                uint32_t b[4];
                key_b(base + L::K + pb * L::kPlane, n * 16, c, b);
#pragma unroll
                for (int pa = 0; pa + pb < NI; ++pa) {
                    ptx::mma16816(kk[2 * n], ak[pa], b[0], b[1]);
                    ptx::mma16816(kk[2 * n + 1], ak[pa], b[2], b[3]);
                    ptx::mma16816(qk[2 * n], aq[pa], b[0], b[1]);
                    ptx::mma16816(qk[2 * n + 1], aq[pa], b[2], b[3]);
                }
            }
        }
    }

    float *A = reinterpret_cast<float *>(smem + L::A);
    float *vec_s = reinterpret_cast<float *>(smem + L::Vec);
    for (int h0 = 0; h0 < group; h0 += 2) {
        const int nh = min(2, group - h0);
        // gates: warp w < nh takes head h0 + w; running sums in double, held as two floats
        if (warp < nh) {
            const int head = kh * group + h0 + warp;
            double s[2];
            float b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane * 2 + i;
                float x = 0.f;
                b[i] = 0.f;
                if (r < ch.len) {
                    x = p.g[(ch.t0 + r) * hv + head];
                    // below -200 (and at -inf) the decay is 0 in fp32 all the same; a finite
                    // floor keeps differences of the sums free of inf - inf
                    x = x < kGFloor ? kGFloor : x;
                    b[i] = p.beta[(ch.t0 + r) * hv + head];
                }
                s[i] = x;
            }
            s[1] += s[0];
            double run = s[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += y;
            }
            const double before = run - s[1], total = __shfl_sync(0xffffffffu, run, 31);
            float *out = reinterpret_cast<float *>(ws + (slot * hv + head) * terms_bytes(NS) + (size_t)2 * NS * kTile * 2);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane * 2 + i;
                const double G = before + s[i];
                const float hi = (float)G, lo = (float)(G - (double)hi);
                vec_s[warp * 3 * C + r] = hi;
                vec_s[warp * 3 * C + C + r] = lo;
                vec_s[warp * 3 * C + 2 * C + r] = b[i];
                out[r] = expf(hi);
                out[C + r] = expf((float)(total - G));
                out[2 * C + r] = b[i];
                out[3 * C + r] = expf((float)total);
                out[4 * C + r] = hi;
                out[5 * C + r] = lo;
            }
        }
        __syncthreads();  // the gates are in; K and Q (or the previous pair's P) are done with
        // A (fp32, zero above the diagonal) and P (bf16 planes) of both heads
        for (int hh = 0; hh < nh; ++hh) {
            const float *Gh = vec_s + hh * 3 * C, *Gl = Gh + C, *B = Gl + C;
            char *tile = smem + hh * L::kHead;
            const int r0 = warp * 16 + (lane >> 2);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const int j = n * 8 + (lane & 3) * 2;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int r = r0 + hf * 8;
                    float a[2], pv[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float d = (Gh[r] - Gh[j + i]) + (Gl[r] - Gl[j + i]);
                        const float e = j + i <= r ? expf(d) : 0.f;
                        pv[i] = j + i <= r ? scale * e * qk[n][hf * 2 + i] : 0.f;
                        a[i] = j + i < r ? B[r] * e * kk[n][hf * 2 + i] : 0.f;
                    }
                    *reinterpret_cast<float2 *>(A + hh * C * kARow + r * kARow + j) = make_float2(a[0], a[1]);
                    uint32_t w[NS];
                    split2<NS>(pv[0], pv[1], w);
#pragma unroll
                    for (int pl = 0; pl < NS; ++pl)
                        *reinterpret_cast<uint32_t *>(tile + pl * kTile * 2 + tile_off<128>(r, j)) = w[pl];
                }
            }
        }
        __syncthreads();
        for (int hh = 0; hh < nh; ++hh) {  // P out
            const int head = kh * group + h0 + hh;
            uint4 *dst = reinterpret_cast<uint4 *>(ws + (slot * hv + head) * terms_bytes(NS) + (size_t)NS * kTile * 2);
            const uint4 *src = reinterpret_cast<const uint4 *>(smem + hh * L::kHead);
            for (int i = tid; i < NS * kTile / 8; i += kTermThreads) dst[i] = src[i];
        }
        // X in place: warps 2 h, 2 h + 1 for head h
        {
            const int hh = warp >> 1, w = warp & 1, t = tid & 63;
            float *X = A + hh * C * kARow;
            diagonal_column(X, t >> 4, t & 15, hh < nh);
            __syncthreads();
            join_blocks<16>(X, 32 * w + 16, 32 * w, 0, hh < nh);
            join_blocks<32>(X, 32, 0, 16 * w, hh < nh);
        }
        for (int hh = 0; hh < nh; ++hh) {  // X out, split into planes on the way
            const int head = kh * group + h0 + hh;
            char *dst = ws + (slot * hv + head) * terms_bytes(NS);
            for (int i = tid; i < C * 8; i += kTermThreads) {
                const int r = i >> 3, c = (i & 7) * 8;
                const float *src = A + hh * C * kARow + r * kARow + c;
                uint32_t w[NS][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t s[NS];
                    const float2 v = *reinterpret_cast<const float2 *>(src + 2 * j);
                    split2<NS>(v.x, v.y, s);
#pragma unroll
                    for (int q = 0; q < NS; ++q) w[q][j] = s[q];
                }
#pragma unroll
                for (int q = 0; q < NS; ++q)
                    *reinterpret_cast<uint4 *>(dst + q * kTile * 2 + tile_off<128>(r, c)) =
                        make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
            }
        }
        __syncthreads();  // A and the gates are free for the next pair
    }
}

template <typename T, int DKP>
__global__ void __launch_bounds__(kChainThreads)
    gdr_chain_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const GdrArgs p, const Images im, float scale,
                     bool wide_out) {
    chain<T, DKP, Mode::kForward>(tm_q, tm_k, tm_v, p, im, 1, blockIdx.x, scale, wide_out);
}

template <typename T, int DKP>
cudaError_t terms(const GdrArgs &p, const Images &im, int values, cudaStream_t stream) {
    constexpr int bytes = TermsSmem<InputPlanes<T>::N, DKP>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(gdr_terms_kernel<T, DKP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const bool vec = rows_vec<T>(p.q, p.q_stride, p.d_k) && rows_vec<T>(p.k, p.k_stride, p.d_k);
    const dim3 grid((unsigned)n_slots(p.n_tok, p.n_seq), p.n_k_heads);
    gdr_terms_kernel<T, DKP><<<grid, kTermThreads, bytes, stream>>>(p, im, values, 1.f / std::sqrt((float)p.d_k), vec);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int DKP>
cudaError_t forward(const GdrArgs &p, cudaStream_t stream) {
    ChainMaps maps;
    Images im{!maps.make<T>(p, false), scan_offset(p.n_tok, p.n_seq, p.n_heads, InputPlanes<T>::N == 1 ? 2 : 3)};
    cudaError_t e = launch_gdr_terms(p, im, 1, stream);
    if (e != cudaSuccess) return e;
    constexpr int bytes = ChainSmem<InputPlanes<T>::N, DKP, Mode::kForward>::kBytes;
    e = cudaFuncSetAttribute(gdr_chain_kernel<T, DKP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const bool wide = p.d_v % 2 == 0 && ((uintptr_t)p.out % (2 * sizeof(T))) == 0;
    gdr_chain_kernel<T, DKP><<<chain_blocks(p), kChainThreads, bytes, stream>>>(
        maps.q, maps.k, maps.v, p, im, 1.f / std::sqrt((float)p.d_k), wide);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace
}  // namespace gdr

size_t gdr_fwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k,
                               int32_t d_v, bool bf16) {
    return gdr::scan_offset(n_tok, n_seq, n_heads, bf16 ? 2 : 3) +
           (size_t)gdr::n_slots(n_tok, n_seq) *
               gdr::Images::record(bf16 ? 1 : 3, d_k <= 64 ? 64 : 128, d_v, n_k_heads, n_heads, 1);
}

cudaError_t launch_gdr_terms(const GdrArgs &p, gdr::Images im, int values, cudaStream_t stream) {
    if (p.n_tok == 0) return cudaSuccess;
    if (p.bf16) return p.d_k <= 64 ? gdr::terms<__nv_bfloat16, 64>(p, im, values, stream) : gdr::terms<__nv_bfloat16, 128>(p, im, values, stream);
    return p.d_k <= 64 ? gdr::terms<float, 64>(p, im, values, stream) : gdr::terms<float, 128>(p, im, values, stream);
}

cudaError_t launch_gdr_fwd(const GdrArgs &p, cudaStream_t stream) {
    if (p.bf16) return p.d_k <= 64 ? gdr::forward<__nv_bfloat16, 64>(p, stream) : gdr::forward<__nv_bfloat16, 128>(p, stream);
    return p.d_k <= 64 ? gdr::forward<float, 64>(p, stream) : gdr::forward<float, 128>(p, stream);
}

cudaError_t read_gdr_fwd_flags(unsigned int *flags, bool reset, cudaStream_t stream) {
    return gdr::read_flags(flags, reset, stream);
}

}  // namespace kda
