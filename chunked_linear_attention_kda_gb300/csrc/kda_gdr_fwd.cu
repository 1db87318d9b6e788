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
    static constexpr int kPlane = C * DKP * 2;
    static constexpr int K = 0, Q = K + NI * kPlane, A = Q + NI * kPlane;
    static constexpr int Vec = A + 2 * C * kARow * 4;          // per head: Ghi, Glo, beta
    static constexpr int Tile = Vec + 2 * 3 * C * 4;
};

// X = (I + A)^-1 column by column: thread j solves for column j by forward substitution, the
// whole column in registers, the rows of A broadcast from shared memory.
__device__ __forceinline__ void solve_column(const float *A, int j, float *x) {
#pragma unroll
    for (int r = 0; r < C; ++r) {
        float s0 = r == j ? 1.f : 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int k = 0; k < (r & ~3); k += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(A + r * kARow + k);
            s0 = fmaf(-a.x, x[k], s0);
            s1 = fmaf(-a.y, x[k + 1], s1);
            s2 = fmaf(-a.z, x[k + 2], s2);
            s3 = fmaf(-a.w, x[k + 3], s3);
        }
#pragma unroll
        for (int k = r & ~3; k < r; ++k) s1 = fmaf(-A[r * kARow + k], x[k], s1);
        x[r] = (s0 + s1) + (s2 + s3);
    }
}

template <typename T, int DKP>
__global__ void __launch_bounds__(kTermThreads)
    gdr_terms_kernel(const T *__restrict__ q, const T *__restrict__ k, int64_t q_stride, int64_t k_stride,
                     const float *__restrict__ g, const float *__restrict__ beta,
                     const int32_t *__restrict__ cu, char *__restrict__ ws, int n_seq, int hk, int hv,
                     int dk, float scale, bool vec) {
    constexpr int NI = InputPlanes<T>::N, NS = NI == 1 ? 2 : 3;
    using L = TermsSmem<NI, DKP>;
    constexpr int RB = DKP * 2;
    extern __shared__ __align__(128) char smem[];
    const uint32_t base = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t slot = blockIdx.x;
    const Chunk ch = find_chunk(cu, n_seq, slot);
    if (ch.len == 0) return;
    const int kh = blockIdx.y, group = hv / hk;

    load_tile<T, RB>(base + L::K, L::kPlane, k + ch.t0 * k_stride + (int64_t)kh * dk, k_stride, ch.len,
                     dk, vec, tid, kTermThreads);
    load_tile<T, RB>(base + L::Q, L::kPlane, q + ch.t0 * q_stride + (int64_t)kh * dk, q_stride, ch.len,
                     dk, vec, tid, kTermThreads);
    ptx::cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();

    // K K^T and Q K^T: warp w the rows 16 w .., columns up to its own
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) kk[n][i] = qk[n][i] = 0.f;
#pragma unroll 1
    for (int c = 0; c < DKP; c += 16) {
        uint32_t ak[NI][4], aq[NI][4];
#pragma unroll
        for (int p = 0; p < NI; ++p) {
            frag_a<RB>(base + L::K + p * L::kPlane, warp * 16, c, ak[p]);
            frag_a<RB>(base + L::Q + p * L::kPlane, warp * 16, c, aq[p]);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n > warp) break;
#pragma unroll
            for (int pb = 0; pb < NI; ++pb) {
                uint32_t b[4];
                frag_b<RB>(base + L::K + pb * L::kPlane, n * 16, c, b);
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
        __syncthreads();  // the previous pair of heads is done with A and the tile
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
                    x = g[(ch.t0 + r) * hv + head];
                    // below -200 (and at -inf) the decay is 0 in fp32 all the same; a finite
                    // floor keeps differences of the sums free of inf - inf
                    x = x < kGFloor ? kGFloor : x;
                    b[i] = beta[(ch.t0 + r) * hv + head];
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
            float *out = reinterpret_cast<float *>(ws + (slot * hv + head) * terms_bytes(NS) +
                                                   (size_t)2 * NS * kTile * 2);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane * 2 + i;
                const double G = before + s[i];
                const float hi = (float)G;
                vec_s[warp * 3 * C + r] = hi;
                vec_s[warp * 3 * C + C + r] = (float)(G - (double)hi);
                vec_s[warp * 3 * C + 2 * C + r] = b[i];
                out[r] = expf(hi);
                out[C + r] = expf((float)(total - G));
                out[2 * C + r] = b[i];
                out[3 * C + r] = expf((float)total);
                out[4 * C + r] = hi;
                out[5 * C + r] = (float)(G - (double)hi);
            }
        }
        __syncthreads();
        // A (fp32) and P (bf16 planes) of both heads
        for (int hh = 0; hh < nh; ++hh) {
            const float *Gh = vec_s + hh * 3 * C, *Gl = Gh + C, *B = Gl + C;
            char *tile = smem + L::Tile + hh * NS * kTile * 2;
            const int r0 = warp * 16 + (lane >> 2);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const int j = n * 8 + (lane & 3) * 2;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int r = r0 + hf * 8;
                    float a[2], p[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float d = (Gh[r] - Gh[j + i]) + (Gl[r] - Gl[j + i]);
                        const float e = j + i <= r ? expf(d) : 0.f;
                        p[i] = j + i <= r ? scale * e * qk[n][hf * 2 + i] : 0.f;
                        a[i] = j + i < r ? B[r] * e * kk[n][hf * 2 + i] : 0.f;
                    }
                    *reinterpret_cast<float2 *>(A + hh * C * kARow + r * kARow + j) = make_float2(a[0], a[1]);
                    uint32_t w[NS];
                    split2<NS>(p[0], p[1], w);
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
            const uint4 *src = reinterpret_cast<const uint4 *>(smem + L::Tile + hh * NS * kTile * 2);
            for (int i = tid; i < NS * kTile / 8; i += kTermThreads) dst[i] = src[i];
        }
        float x[C];
        const int hh = warp >> 1, j = tid & (C - 1);
        if (hh < nh) solve_column(A + hh * C * kARow, j, x);
        __syncthreads();
        if (hh < nh) {
            char *tile = smem + L::Tile + hh * NS * kTile * 2;
#pragma unroll
            for (int r = 0; r < C; ++r) {
                float v = x[r];
#pragma unroll
                for (int pl = 0; pl < NS; ++pl) {
                    const __nv_bfloat16 b = __float2bfloat16_rn(v);
                    *reinterpret_cast<__nv_bfloat16 *>(tile + pl * kTile * 2 + tile_off<128>(r, j)) = b;
                    v -= __bfloat162float(b);
                }
            }
        }
        __syncthreads();
        for (int hx = 0; hx < nh; ++hx) {  // X out
            const int head = kh * group + h0 + hx;
            uint4 *dst = reinterpret_cast<uint4 *>(ws + (slot * hv + head) * terms_bytes(NS));
            const uint4 *src = reinterpret_cast<const uint4 *>(smem + L::Tile + hx * NS * kTile * 2);
            for (int i = tid; i < NS * kTile / 8; i += kTermThreads) dst[i] = src[i];
        }
    }
}

template <typename T, int DKP, int W>
__global__ void __launch_bounds__(32 * W)
    gdr_chain_kernel(const GdrArgs p, float scale, bool vec_qk, bool vec_v, bool wide_out) {
    chain<T, DKP, W, false>(p, blockIdx.x, scale, vec_qk, vec_v, wide_out);
}

template <typename T, int DKP>
cudaError_t terms(const GdrArgs &p, cudaStream_t stream) {
    constexpr int NI = InputPlanes<T>::N, NS = NI == 1 ? 2 : 3;
    constexpr int bytes = TermsSmem<NI, DKP>::Tile + 2 * NS * kTile * 2;
    const cudaError_t e = cudaFuncSetAttribute(gdr_terms_kernel<T, DKP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const bool vec = rows_vec<T>(p.q, p.q_stride, p.d_k) && rows_vec<T>(p.k, p.k_stride, p.d_k);
    const dim3 grid((unsigned)n_slots(p.n_tok, p.n_seq), p.n_k_heads);
    gdr_terms_kernel<T, DKP><<<grid, kTermThreads, bytes, stream>>>(
        static_cast<const T *>(p.q), static_cast<const T *>(p.k), p.q_stride, p.k_stride, p.g, p.beta,
        p.cu_seqlens, static_cast<char *>(p.workspace), p.n_seq, p.n_k_heads, p.n_heads, p.d_k,
        1.f / std::sqrt((float)p.d_k), vec);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int DKP>
cudaError_t forward(const GdrArgs &p, cudaStream_t stream) {
    constexpr int W = 2;
    using L = ChainSmem<InputPlanes<T>::N, DKP, W, false>;
    const cudaError_t e = cudaFuncSetAttribute(gdr_chain_kernel<T, DKP, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    if (e != cudaSuccess) return e;
    const bool vec_qk = rows_vec<T>(p.q, p.q_stride, p.d_k) && rows_vec<T>(p.k, p.k_stride, p.d_k);
    const bool vec_v = rows_vec<T>(p.v, p.v_stride, p.d_v);
    const bool wide = p.d_v % 2 == 0 && ((uintptr_t)p.out % (2 * sizeof(T))) == 0;
    const unsigned grid = (unsigned)((p.d_v + 16 * W - 1) / (16 * W)) * p.n_heads * p.n_seq;
    gdr_chain_kernel<T, DKP, W><<<grid, 32 * W, L::kBytes, stream>>>(p, 1.f / std::sqrt((float)p.d_k), vec_qk, vec_v, wide);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace
}  // namespace gdr

size_t gdr_fwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, bool bf16) {
    return (size_t)gdr::n_slots(n_tok, n_seq) * n_heads * gdr::terms_bytes(bf16 ? 2 : 3);
}

cudaError_t launch_gdr_terms(const GdrArgs &p, cudaStream_t stream) {
    if (p.n_tok == 0) return cudaSuccess;
    if (p.bf16) return p.d_k <= 64 ? gdr::terms<__nv_bfloat16, 64>(p, stream) : gdr::terms<__nv_bfloat16, 128>(p, stream);
    return p.d_k <= 64 ? gdr::terms<float, 64>(p, stream) : gdr::terms<float, 128>(p, stream);
}

cudaError_t launch_gdr_fwd(const GdrArgs &p, cudaStream_t stream) {
    const cudaError_t e = launch_gdr_terms(p, stream);
    if (e != cudaSuccess) return e;
    if (p.bf16) return p.d_k <= 64 ? gdr::forward<__nv_bfloat16, 64>(p, stream) : gdr::forward<__nv_bfloat16, 128>(p, stream);
    return p.d_k <= 64 ? gdr::forward<float, 64>(p, stream) : gdr::forward<float, 128>(p, stream);
}

}  // namespace kda
