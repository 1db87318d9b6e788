// The serial chain over a sequence's chunks (see kda_gdr_fwd.cu), used by the forward pass
// and, without its output, by the backward pass. Internal; not part of the C ABI.
#pragma once

#include "kda_gdr.h"

namespace kda {
namespace gdr {

template <int NI, int DKP, int W, bool STATES>
struct ChainSmem {
    static constexpr int NS = NI == 1 ? 2 : 3;
    static constexpr int NP = NI;              // planes of P read for the output
    static constexpr int kStages = NI == 1 ? 2 : 1;
    static constexpr int kPlane = C * DKP * 2, kVPlane = C * 16 * W * 2;
    static constexpr int K = 0, X = K + NI * kPlane, Gate = X + NS * kTile * 2, V = Gate + kChainGates * 4;
    static constexpr int Q = V + NI * kVPlane, P = Q + (STATES ? 0 : NI * kPlane);
    static constexpr int kStage = P + (STATES ? 0 : NP * kTile * 2);
    static constexpr int kBytes = kStages * kStage;
};

// One CTA's chain: 16 W value channels of one (sequence, head), `block` counting channel
// blocks, then heads, then sequences. STATES: no output; every chunk's S0^T and U^T go to
// the workspace instead.
template <typename T, int DKP, int W, bool STATES>
__device__ __forceinline__ void chain(const GdrArgs &p, int block, float scale, bool vec_qk, bool vec_v, bool wide_out) {
    constexpr int NI = InputPlanes<T>::N;
    using L = ChainSmem<NI, DKP, W, STATES>;
    constexpr int NS = L::NS, RB = DKP * 2, VB = 32 * W, NT = DKP / 8;
    extern __shared__ __align__(128) char smem[];
    const uint32_t base = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tq = lane & 3;
    const int n_blk = (p.d_v + 16 * W - 1) / (16 * W);
    const int blk = block % n_blk, sh = block / n_blk;
    const int head = sh % p.n_heads, seq = sh / p.n_heads, kh = head / (p.n_heads / p.n_k_heads);
    const int64_t tok0 = p.cu_seqlens[seq];
    const int len = (int)(p.cu_seqlens[seq + 1] - tok0);
    const int n_chunks = (len + C - 1) / C;
    const int64_t slot0 = slot_base(p.cu_seqlens, seq);
    const int dv0 = blk * 16 * W, v0 = dv0 + warp * 16;
    const char *terms = static_cast<const char *>(p.workspace) + (slot0 * p.n_heads + head) * terms_bytes(NS);
    const size_t terms_step = (size_t)p.n_heads * terms_bytes(NS);

    // S^T: tile n holds rows (value channels) gr, gr + 8 and columns (key channels) 8 n + 2 tq, + 1
    float S[NT][4];
    const size_t st_at = ((size_t)seq * p.n_heads + head) * p.d_k * p.d_v;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = n * 8 + tq * 2 + (i & 1), v = v0 + gr + (i >> 1) * 8;
            S[n][i] = p.h0 && c < p.d_k && v < p.d_v ? p.h0[st_at + (size_t)c * p.d_v + v] : 0.f;
        }

    auto load = [&](int c) {
        const uint32_t s = base + (c % L::kStages) * L::kStage;
        const int64_t t = tok0 + (int64_t)c * C;
        const int rows = min(C, len - c * C);
        load_tile<T, RB>(s + L::K, L::kPlane, static_cast<const T *>(p.k) + t * p.k_stride + (int64_t)kh * p.d_k,
                         p.k_stride, rows, p.d_k, vec_qk, tid, 32 * W);
        if (!STATES) load_tile<T, RB>(s + L::Q, L::kPlane, static_cast<const T *>(p.q) + t * p.q_stride + (int64_t)kh * p.d_k,
                         p.q_stride, rows, p.d_k, vec_qk, tid, 32 * W);
        load_tile<T, VB>(s + L::V, L::kVPlane,
                         static_cast<const T *>(p.v) + t * p.v_stride + (int64_t)head * p.d_v + dv0, p.v_stride,
                         rows, p.d_v - dv0, vec_v, tid, 32 * W);
        const char *src = terms + c * terms_step;
        load_raw(s + L::X, src, NS * kTile * 2, tid, 32 * W);
        if (!STATES) load_raw(s + L::P, src + NS * kTile * 2, L::NP * kTile * 2, tid, 32 * W);
        load_raw(s + L::Gate, src + 2 * NS * kTile * 2, kChainGates * 4, tid, 32 * W);
    };

    if (L::kStages == 2 && n_chunks > 0) load(0);
    ptx::cp_async_commit();
    for (int c = 0; c < n_chunks; ++c) {
        if (L::kStages == 2) {
            if (c + 1 < n_chunks) load(c + 1);
            ptx::cp_async_commit();
            cp_async_wait<1>();
        } else {
            load(c);
            ptx::cp_async_commit();
            cp_async_wait<0>();
        }
        __syncthreads();
        const uint32_t s = base + (c % L::kStages) * L::kStage;
        const float *gate = reinterpret_cast<const float *>(smem + (c % L::kStages) * L::kStage + L::Gate);

        [[maybe_unused]] char *rec = nullptr;  // this chunk's record of the scan
        if constexpr (STATES) {
            rec = static_cast<char *>(p.workspace) + scan_offset(p.n_tok, p.n_seq, p.n_heads, NS) +
                  ((slot0 + c) * p.n_heads + head) * scan_bytes(NS, DKP, p.d_v);
            if (v0 < pad_v(p.d_v)) store_planes<NS, NT, RB>(rec, (size_t)pad_v(p.d_v) * RB, v0, S);
        }
        // Y^T = S^T K^T
        float y[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[n][i] = 0.f;
#pragma unroll
        for (int kx = 0; kx < DKP / 16; ++kx) {
            uint32_t a[NS][4];
            acc_to_a<NS>(&S[2 * kx], a);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int pb = 0; pb < NI; ++pb) {
                    uint32_t b[4];
                    frag_b<RB>(s + L::K + pb * L::kPlane, n * 16, kx * 16, b);
#pragma unroll
                    for (int pa = 0; pa + pb < NS; ++pa) {
                        ptx::mma16816(y[2 * n], a[pa], b[0], b[1]);
                        ptx::mma16816(y[2 * n + 1], a[pa], b[2], b[3]);
                    }
                }
        }
        // beta Z^T = beta (V^T - gamma Y^T), in place
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
            for (int pl = 0; pl < NI; ++pl) {
                uint32_t w[4];
                ptx::ldsm_x4_t(s + L::V + pl * L::kVPlane +
                                   tile_off<VB>(n * 16 + (lane >> 4) * 8 + (lane & 7), warp * 16 + ((lane >> 3) & 1) * 8),
                               w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] += lo_f(w[i]);
                    v[2 * i + 1] += hi_f(w[i]);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = n * 16 + h * 8 + tq * 2;
                const float2 ga = *reinterpret_cast<const float2 *>(gate + t);
                const float2 be = *reinterpret_cast<const float2 *>(gate + 2 * C + t);
                float *z = y[2 * n + h];
                z[0] = be.x * fmaf(-ga.x, z[0], v[4 * h]);
                z[1] = be.y * fmaf(-ga.y, z[1], v[4 * h + 1]);
                z[2] = be.x * fmaf(-ga.x, z[2], v[4 * h + 2]);
                z[3] = be.y * fmaf(-ga.y, z[3], v[4 * h + 3]);
            }
        }
        // U^T = (beta Z)^T X^T, X lower triangular
        float u[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) u[n][i] = 0.f;
#pragma unroll
        for (int kx = 0; kx < 4; ++kx) {
            uint32_t a[NS][4];
            acc_to_a<NS>(&y[2 * kx], a);
#pragma unroll
            for (int n = kx; n < 4; ++n)
#pragma unroll
                for (int pb = 0; pb < NS; ++pb) {
                    uint32_t b[4];
                    frag_b<128>(s + L::X + pb * kTile * 2, n * 16, kx * 16, b);
#pragma unroll
                    for (int pa = 0; pa + pb < NS; ++pa) {
                        ptx::mma16816(u[2 * n], a[pa], b[0], b[1]);
                        ptx::mma16816(u[2 * n + 1], a[pa], b[2], b[3]);
                    }
                }
        }
        if constexpr (STATES) {
            if (v0 < pad_v(p.d_v)) store_planes<NS, 8, 128>(rec + 2 * scan_state_bytes(NS, DKP, p.d_v), (size_t)pad_v(p.d_v) * 128, v0, u);
        } else {  // O = scale gamma Q S0 + (scale P) U, tokens on the rows
            float o[4][2][4];
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[m][n][i] = 0.f;
#pragma unroll
            for (int kx = 0; kx < DKP / 16; ++kx) {
                uint32_t a[NI][4];
                acc_to_a<NI>(&S[2 * kx], a);
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int pq = 0; pq < NI; ++pq) {
                        uint32_t f[4];
                        frag_a<RB>(s + L::Q + pq * L::kPlane, m * 16, kx * 16, f);
#pragma unroll
                        for (int pa = 0; pa + pq < NI; ++pa) {
                            ptx::mma16816(o[m][0], f, a[pa][0], a[pa][2]);
                            ptx::mma16816(o[m][1], f, a[pa][1], a[pa][3]);
                        }
                    }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float g0 = scale * gate[m * 16 + gr], g1 = scale * gate[m * 16 + gr + 8];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    o[m][n][0] *= g0; o[m][n][1] *= g0; o[m][n][2] *= g1; o[m][n][3] *= g1;
                }
            }
#pragma unroll
            for (int kx = 0; kx < 4; ++kx) {
                uint32_t a[NS][4];
                acc_to_a<NS>(&u[2 * kx], a);
#pragma unroll
                for (int m = kx; m < 4; ++m)
#pragma unroll
                    for (int pq = 0; pq < L::NP; ++pq) {
                        uint32_t f[4];
                        frag_a<128>(s + L::P + pq * kTile * 2, m * 16, kx * 16, f);
#pragma unroll
                        for (int pa = 0; pa + pq < NS; ++pa) {
                            ptx::mma16816(o[m][0], f, a[pa][0], a[pa][2]);
                            ptx::mma16816(o[m][1], f, a[pa][1], a[pa][3]);
                        }
                    }
            }
            T *out = static_cast<T *>(p.out);
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int r = c * C + m * 16 + gr + hf * 8;
                    if (r >= len) continue;
                    T *row = out + ((tok0 + r) * p.n_heads + head) * p.d_v;
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int v = v0 + n * 8 + tq * 2;
                        if (v < p.d_v) put2(row + v, o[m][n][hf * 2], o[m][n][hf * 2 + 1], wide_out, v + 1 < p.d_v);
                    }
                }
        }
        // S1^T = Gamma S0^T + (delta U)^T K
        const float whole = gate[3 * C];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[n][i] *= whole;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 de = *reinterpret_cast<const float2 *>(gate + C + n * 8 + tq * 2);
            u[n][0] *= de.x; u[n][1] *= de.y; u[n][2] *= de.x; u[n][3] *= de.y;
        }
#pragma unroll
        for (int kx = 0; kx < 4; ++kx) {
            uint32_t a[NS][4];
            acc_to_a<NS>(&u[2 * kx], a);
#pragma unroll
            for (int n = 0; n < DKP / 16; ++n)
#pragma unroll
                for (int pb = 0; pb < NI; ++pb) {
                    uint32_t b[4];
                    frag_b_t<RB>(s + L::K + pb * L::kPlane, kx * 16, n * 16, b);
#pragma unroll
                    for (int pa = 0; pa + pb < NS; ++pa) {
                        ptx::mma16816(S[2 * n], a[pa], b[0], b[1]);
                        ptx::mma16816(S[2 * n + 1], a[pa], b[2], b[3]);
                    }
                }
        }
        __syncthreads();
    }
    if (!STATES && p.h_final) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = n * 8 + tq * 2 + (i & 1), v = v0 + gr + (i >> 1) * 8;
                if (c < p.d_k && v < p.d_v) p.h_final[st_at + (size_t)c * p.d_v + v] = S[n][i];
            }
    }
}

}  // namespace gdr
}  // namespace kda
