// The serial chains over a sequence's chunks: the forward's (with its output, or for the
// backward pass with a record of every chunk's state) and the backward's reverse one. The
// mathematics is in kda_gdr_fwd.cu and kda_gdr_bwd.cu. Internal; not part of the C ABI.
//
// A CTA advances 32 value channels of one (sequence, head) through the sequence:
//   warps 0, 1  the state: 16 value channels each, S^T (16 x d_k, fp32) in registers for the
//               whole sequence. An fp32 accumulator tile of mma.sync lies in registers as the
//               A operand (and as the B operand of the transposed product) of the next one,
//               so S^T -> Y^T -> Z^T -> U^T -> S^T never leaves the warp: the serial path
//               has no barrier and no shared-memory round trip.
//   warps 2, 3  what the serial path need not wait for: the output O (from copies of S^T and
//               U^T handed over in shared memory) or, in reverse, dO^T P and (gamma dO)^T Q,
//               which they hand to the state warps ahead of their use.
//   warp 4      one thread loads: tensor copies of whole chunks, bulk copies of the chunk
//               terms and of tile images, into rings of stages (one ring for what the state
//               warps read, one for the others').
// Per chunk and state warp (bf16, d_k = 128) 316 mma.sync m16n8k16 at 8 cycles each bound a
// step from below: 1.3 us.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_gdr.h"

namespace kda {
namespace gdr {

enum class Mode { kForward, kStates, kReverse };
constexpr int kChainThreads = 160;
constexpr int kBlockV = 32;  // value channels of a CTA
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
__device__ __forceinline__ void bulk_wait0() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Shared memory (offsets from a 1024-byte boundary). Ring 1 (state warps): K, X, gates and,
// forward, V. Ring 2 (the others): Q, P, gates and, reverse, dO. Hand: from the state warps
// to the others (forward: S^T and U^T fragments) or back (reverse: two accumulators). Keep:
// the state warps' staging of the records that go to the workspace.
template <int NI, int DKP, Mode M>
struct ChainSmem {
    static constexpr int NS = NI == 1 ? 2 : 3;
    static constexpr bool kOut = M == Mode::kForward, kRev = M == Mode::kReverse;
    static constexpr int kKey = NI * C * DKP * 2, kVal = NI * C * kBlockV * 2;
    static constexpr int kX = NS * kTile * 2;
    static constexpr int kP = (kOut ? NI : NS) * kTile * 2;       // the output takes P in bf16 for bf16
    static constexpr int kGate = kChainGates * 4;
    // ring 1
    static constexpr int K = 0, V = K + kKey, X = V + (kRev ? 0 : kVal), Gate1 = X + kX;
    static constexpr int kStage1 = Gate1 + kGate;
    static constexpr int kBytes1 = kStage1;
    static constexpr int N1 = NI == 1 ? (kRev ? 2 : 3) : 1;
    // ring 2
    static constexpr int Q = 0, dO = Q + kKey, P = dO + (kRev ? kVal : 0), Gate2 = P + kP;
    static constexpr int kStage2 = Gate2 + kGate;
    static constexpr int N2 = M == Mode::kStates ? 0 : NI == 1 ? 2 : 1;
    // per warp
    static constexpr int NH = NI == 1 ? 2 : 1;                    // hand-over buffers
    static constexpr int kHandS = kOut ? NI * DKP * 32 : DKP * 64;       // S^T fragments, or G^T accumulators
    static constexpr int kHandU = kOut ? NS * C * 32 : C * 64;           // U^T fragments, or (dO^T P) accumulators
    static constexpr int kHand = M == Mode::kStates ? 0 : kHandS + kHandU;
    static constexpr int kKeepS = NS * 16 * DKP * 2, kKeepU = NS * 16 * C * 2;
    static constexpr int kKeep = kOut ? 0 : kKeepS + kKeepU;
    static constexpr int Ring2 = N1 * kStage1, Hand = Ring2 + N2 * kStage2, Keep = Hand + 2 * NH * kHand;
    static constexpr int Bars = Keep + 2 * kKeep;
    static constexpr int kBars = 2 * N1 + 2 * N2 + 4 * NH;
    static constexpr int kBytes = Bars + 8 * kBars + 1024;        // the base is rounded up to 1024
    static_assert(kBytes <= 227 * 1024, "fits an SM");
    static_assert(kStage1 % 1024 == 0 && kStage2 % 1024 == 0, "tensor copies land on swizzle boundaries");
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
        if (sizeof(T) != 2 || p.n_tok < C) return false;
        if (!rows_vec<T>(p.q, p.q_stride, p.d_k) || !rows_vec<T>(p.k, p.k_stride, p.d_k) ||
            !rows_vec<T>(p.v, p.v_stride, p.d_v))
            return false;
        const int64_t vs = (int64_t)p.n_heads * p.d_v;
        if (with_dout && !rows_vec<T>(p.dout, vs, p.d_v)) return false;
        return encode(&q, p.q, p.n_tok, p.q_stride, p.n_k_heads, p.d_k, 64) &&
               encode(&k, p.k, p.n_tok, p.k_stride, p.n_k_heads, p.d_k, 64) &&
               encode(&v, p.v, p.n_tok, p.v_stride, p.n_heads, p.d_v, kBlockV) &&
               (!with_dout || encode(&dout, p.dout, p.n_tok, vs, p.n_heads, p.d_v, kBlockV));
    }
};

inline unsigned chain_blocks(const GdrArgs &p) {
    return (unsigned)((p.d_v + kBlockV - 1) / kBlockV) * p.n_heads * p.n_seq;
}

// The sequence of the given rank, longest first (ties by index): the longest chains start
// first. Beyond 1024 sequences they are taken in order.
__device__ __forceinline__ int ranked_sequence(const int32_t *cu, int n_seq, int rank, int *shared) {
    if (n_seq == 1 || n_seq > 1024) return rank;
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

// ---- products of the state warps: S is NT tiles of S^T (rows: 16 value channels)

// y (16 x 64) += S^T K^T
template <int NI, int NS, int DKP>
__device__ __forceinline__ void state_times_keys(const float (*S)[4], uint32_t k, float (*y)[4]) {
#pragma unroll
    for (int kx = 0; kx < DKP / 16; ++kx) {
        uint32_t a[NS][4];
        acc_to_a<NS>(&S[2 * kx], a);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int pb = 0; pb < NI; ++pb) {
                uint32_t b[4];
                key_b(k + pb * C * DKP * 2, n * 16, kx * 16, b);
#pragma unroll
                for (int pa = 0; pa + pb < NS; ++pa) {
                    ptx::mma16816(y[2 * n], a[pa], b[0], b[1]);
                    ptx::mma16816(y[2 * n + 1], a[pa], b[2], b[3]);
                }
            }
    }
}
// S += u^T K, u^T (16 x 64) an accumulator
template <int NI, int NS, int DKP>
__device__ __forceinline__ void add_values_keys(const float (*u)[4], uint32_t k, float (*S)[4]) {
#pragma unroll
    for (int kx = 0; kx < 4; ++kx) {
        uint32_t a[NS][4];
        acc_to_a<NS>(&u[2 * kx], a);
#pragma unroll
        for (int n = 0; n < DKP / 16; ++n)
#pragma unroll
            for (int pb = 0; pb < NI; ++pb) {
                uint32_t b[4];
                key_b_t(k + pb * C * DKP * 2, kx * 16, n * 16, b);
#pragma unroll
                for (int pa = 0; pa + pb < NS; ++pa) {
                    ptx::mma16816(S[2 * n], a[pa], b[0], b[1]);
                    ptx::mma16816(S[2 * n + 1], a[pa], b[2], b[3]);
                }
            }
    }
}
template <int N>
__device__ __forceinline__ void zero(float (*x)[4]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = 0.f;
}
// x (16 x 64, columns = tokens) *= the tokens' factors
__device__ __forceinline__ void scale_tokens(float (*x)[4], const float *f) {
    const int tq = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        const float2 v = *reinterpret_cast<const float2 *>(f + n * 8 + tq * 2);
        x[n][0] *= v.x; x[n][1] *= v.y; x[n][2] *= v.x; x[n][3] *= v.y;
    }
}
template <int NT>
__device__ __forceinline__ void load_state(float (*S)[4], const float *src, int v0, int d_k, int d_v) {
    const int gr = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = n * 8 + tq * 2 + (i & 1), v = v0 + gr + (i >> 1) * 8;
            S[n][i] = src && c < d_k && v < d_v ? src[(size_t)c * d_v + v] : 0.f;
        }
}
template <int NT>
__device__ __forceinline__ void store_state(const float (*S)[4], float *dst, int v0, int d_k, int d_v) {
    const int gr = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = n * 8 + tq * 2 + (i & 1), v = v0 + gr + (i >> 1) * 8;
            if (c < d_k && v < d_v) dst[(size_t)c * d_v + v] = S[n][i];
        }
}

// One CTA's chain; `block` counts channel blocks, then heads, then sequences (longest first).
// tm_v is dout's map in reverse; `values` and `im` as given to the chunk terms.
template <typename T, int DKP, Mode M>
__device__ __forceinline__ void chain(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                      const GdrArgs &p, const Images &im, int values, int block, float scale,
                                      bool wide_out) {
    constexpr int NI = InputPlanes<T>::N;
    using L = ChainSmem<NI, DKP, M>;
    constexpr int NS = L::NS, NT = DKP / 8, N1 = L::N1, N2 = L::N2, NH = L::NH;
    constexpr bool kOut = L::kOut, kRev = L::kRev;
    extern __shared__ __align__(1024) char smem_raw[];
    char *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    __shared__ int ranked;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tq = lane & 3;
    const int n_blk = (p.d_v + kBlockV - 1) / kBlockV;
    const int blk = block % n_blk, sh = block / n_blk;
    const int head = sh % p.n_heads, kh = head / (p.n_heads / p.n_k_heads);
    const int seq = ranked_sequence(p.cu_seqlens, p.n_seq, sh / p.n_heads, &ranked);
    const int64_t tok0 = p.cu_seqlens[seq];
    const int len = (int)(p.cu_seqlens[seq + 1] - tok0);
    const int n_chunks = (len + C - 1) / C;
    const int64_t slot0 = slot_base(p.cu_seqlens, seq);
    const int w = warp & 1, v0 = blk * kBlockV + w * 16;
    const size_t st_at = ((size_t)seq * p.n_heads + head) * p.d_k * p.d_v;
    char *ws = static_cast<char *>(p.workspace);

    auto bar = [&](int i) { return base + L::Bars + 8 * i; };
    auto full1 = [&](int s) { return bar(s); };
    auto empty1 = [&](int s) { return bar(N1 + s); };
    auto full2 = [&](int s) { return bar(2 * N1 + s); };
    auto empty2 = [&](int s) { return bar(2 * N1 + N2 + s); };
    auto hfull = [&](int b) { return bar(2 * N1 + 2 * N2 + b * 2 + w); };
    auto hempty = [&](int b) { return bar(2 * N1 + 2 * N2 + 2 * NH + b * 2 + w); };
    if (tid == 0) {
        for (int s = 0; s < N1; ++s) { ptx::mbar_init(full1(s), 1); ptx::mbar_init(empty1(s), 2); }
        for (int s = 0; s < N2; ++s) { ptx::mbar_init(full2(s), 1); ptx::mbar_init(empty2(s), 2); }
        for (int b = 0; b < 4 * NH; ++b) ptx::mbar_init(bar(2 * N1 + 2 * N2 + b), 1);
        ptx::mbar_init_fence();
    }
    __syncthreads();
    // step i works on chunk at(i)
    auto at = [&](int i) { return kRev ? n_chunks - 1 - i : i; };

    if (warp == 4) {
        // ------------------------------------------------ loads
        if (lane == 0) {
            const size_t rec = Images::record(NI, DKP, p.d_v, p.n_k_heads, p.n_heads, values);
            const size_t kb = Images::key_bytes(NI, DKP), vb = Images::value_bytes(NI, p.d_v);
            int done1 = 0, done2 = 0;
            bool ok = true;
            for (int i = 0; i < n_chunks && ok; ++i) {
                const int c = at(i), t = (int)tok0 + c * C;
                const bool image = im.all || len - c * C < C;
                const char *img = ws + im.offset + (im.all ? slot0 + c : (int64_t)seq) * rec;
                const char *vimg = img + 2 * p.n_k_heads * kb + (kRev ? p.n_heads + head : head) * vb + (size_t)blk * L::kVal;
                const char *terms = ws + ((slot0 + c) * p.n_heads + head) * terms_bytes(NS);
                {
                    const int s = i % N1;
                    const uint32_t d = base + s * L::kStage1, m = full1(s);
                    if (!(ok = wait_bar(empty1(s), ((i / N1) & 1) ^ 1))) break;
                    ptx::mbar_arrive_tx(m, L::kKey + (kRev ? 0 : L::kVal) + L::kX + L::kGate);
                    if (image) {
                        bulk_load(d + L::K, img + (p.n_k_heads + kh) * kb, L::kKey, m);
                        if (!kRev) bulk_load(d + L::V, vimg, L::kVal, m);
                    } else {
#pragma unroll
                        for (int h = 0; h < DKP / 64; ++h) ptx::tma_load_3d(d + L::K + h * kHalf, &tm_k, h * 64, kh, t, m);
                        if (!kRev) ptx::tma_load_3d(d + L::V, &tm_v, blk * kBlockV, head, t, m);
                    }
                    bulk_load(d + L::X, terms, L::kX, m);
                    bulk_load(d + L::Gate1, terms + 2 * NS * kTile * 2, L::kGate, m);
                    ++done1;
                }
                if constexpr (N2 > 0) {
                    const int s = i % N2;
                    const uint32_t d = base + L::Ring2 + s * L::kStage2, m = full2(s);
                    if (!(ok = wait_bar(empty2(s), ((i / N2) & 1) ^ 1))) break;
                    ptx::mbar_arrive_tx(m, L::kKey + (kRev ? L::kVal : 0) + L::kP + L::kGate);
                    if (image) {
                        bulk_load(d + L::Q, img + kh * kb, L::kKey, m);
                        if (kRev) bulk_load(d + L::dO, vimg, L::kVal, m);
                    } else {
#pragma unroll
                        for (int h = 0; h < DKP / 64; ++h) ptx::tma_load_3d(d + L::Q + h * kHalf, &tm_q, h * 64, kh, t, m);
                        if (kRev) ptx::tma_load_3d(d + L::dO, &tm_v, blk * kBlockV, head, t, m);
                    }
                    bulk_load(d + L::P, terms + NS * kTile * 2, L::kP, m);
                    bulk_load(d + L::Gate2, terms + 2 * NS * kTile * 2, L::kGate, m);
                    ++done2;
                }
            }
            if (!ok) {  // nothing may land in shared memory after the CTA has gone
                for (int i = max(0, done1 - N1); i < done1; ++i) wait_bar(full1(i % N1), (i / N1) & 1);
                if constexpr (N2 > 0)
                    for (int i = max(0, done2 - N2); i < done2; ++i) wait_bar(full2(i % N2), (i / N2) & 1);
            }
        }
    } else if (warp < 2) {
        // ------------------------------------------------ state
        float S[NT][4];
        load_state<NT>(S, kRev ? (p.dh_final ? p.dh_final + st_at : nullptr) : (p.h0 ? p.h0 + st_at : nullptr), v0,
                       p.d_k, p.d_v);
        char *keep = smem + L::Keep + w * L::kKeep;
        for (int i = 0; i < n_chunks; ++i) {
            const int c = at(i), s1 = i % N1, hb = i % NH;
            const uint32_t s = base + s1 * L::kStage1;
            const float *gate = reinterpret_cast<const float *>(smem + s1 * L::kStage1 + L::Gate1);
            char *hand = smem + L::Hand + (hb * 2 + w) * L::kHand;
            [[maybe_unused]] char *rec = ws + scan_offset(p.n_tok, p.n_seq, p.n_heads, NS) +
                                         ((slot0 + c) * p.n_heads + head) * scan_bytes(NS, DKP, p.d_v);
            const size_t rec_s = scan_state_bytes(NS, DKP, p.d_v), rec_u = scan_value_bytes(NS, p.d_v);
            const size_t plane_s = (size_t)pad_v(p.d_v) * DKP * 2, plane_u = (size_t)pad_v(p.d_v) * C * 2;
            if (kOut) {  // the others are done with the hand-over of NH steps ago
                if (!warp_wait(hempty(hb), ((i / NH) & 1) ^ 1)) break;
#pragma unroll
                for (int kx = 0; kx < DKP / 16; ++kx) {
                    uint32_t a[NI][4];
                    acc_to_a<NI>(&S[2 * kx], a);
#pragma unroll
                    for (int q = 0; q < NI; ++q)
                        *reinterpret_cast<uint4 *>(hand + ((q * (DKP / 16) + kx) * 32 + lane) * 16) =
                            make_uint4(a[q][0], a[q][1], a[q][2], a[q][3]);
                }
            } else {     // record the chunk's S0 (or dS1); the staging of the last step has been read
                if (lane == 0) ptx::bulk_wait_read0();
                __syncwarp();
                store_planes<NS, NT, DKP * 2>(keep, 16 * DKP * 2, 0, S);
                ptx::fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int q = 0; q < NS; ++q)
                        bulk_store(rec + (kRev ? rec_s : 0) + q * plane_s + (size_t)v0 * DKP * 2,
                                   ptx::smem_u32(keep) + q * 16 * DKP * 2, 16 * DKP * 2);
                    ptx::bulk_commit();
                }
            }
            if (!warp_wait(full1(s1), (i / N1) & 1)) break;

            float y[8][4], u[8][4];
            zero<8>(y);
            zero<8>(u);
            state_times_keys<NI, NS, DKP>(S, s + L::K, y);
            if (!kRev) {
                // beta Z^T = beta (V^T - gamma Y^T), then U^T = (beta Z)^T X^T, X lower triangular
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll
                    for (int q = 0; q < NI; ++q) {
                        uint32_t x[4];
                        ptx::ldsm_x4_t(s + L::V + q * C * kBlockV * 2 +
                                           tile_off<64>(n * 16 + (lane >> 4) * 8 + (lane & 7), w * 16 + ((lane >> 3) & 1) * 8),
                                       x[0], x[1], x[2], x[3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[2 * j] += lo_f(x[j]);
                            v[2 * j + 1] += hi_f(x[j]);
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
            } else {
                // dU^T = delta (dS1^T K^T) + dO^T P, then E^T = dU^T X
                scale_tokens(y, gate + C);
                if (!warp_wait(hfull(hb), (i / NH) & 1)) break;
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float4 x = *reinterpret_cast<const float4 *>(hand + L::kHandS + (n * 32 + lane) * 16);
                    y[n][0] += x.x; y[n][1] += x.y; y[n][2] += x.z; y[n][3] += x.w;
                }
#pragma unroll
                for (int kx = 0; kx < 4; ++kx) {
                    uint32_t a[NS][4];
                    acc_to_a<NS>(&y[2 * kx], a);
#pragma unroll
                    for (int n = 0; n <= kx; ++n)
#pragma unroll
                        for (int pb = 0; pb < NS; ++pb) {
                            uint32_t b[4];
                            frag_b_t<128>(s + L::X + pb * kTile * 2, kx * 16, n * 16, b);
#pragma unroll
                            for (int pa = 0; pa + pb < NS; ++pa) {
                                ptx::mma16816(u[2 * n], a[pa], b[0], b[1]);
                                ptx::mma16816(u[2 * n + 1], a[pa], b[2], b[3]);
                            }
                        }
                }
            }
            // hand U^T over, or record it (E^T)
            if (kOut) {
#pragma unroll
                for (int kx = 0; kx < 4; ++kx) {
                    uint32_t a[NS][4];
                    acc_to_a<NS>(&u[2 * kx], a);
#pragma unroll
                    for (int q = 0; q < NS; ++q)
                        *reinterpret_cast<uint4 *>(hand + L::kHandS + ((q * 4 + kx) * 32 + lane) * 16) =
                            make_uint4(a[q][0], a[q][1], a[q][2], a[q][3]);
                }
                warp_arrive(hfull(hb));
            } else {
                char *ku = keep + L::kKeepS;
                store_planes<NS, 8, 128>(ku, 16 * C * 2, 0, u);
                ptx::fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int q = 0; q < NS; ++q)
                        bulk_store(rec + 2 * rec_s + (kRev ? rec_u : 0) + q * plane_u + (size_t)v0 * C * 2,
                                   ptx::smem_u32(ku) + q * 16 * C * 2, 16 * C * 2);
                    ptx::bulk_commit();
                }
            }
            const float whole = gate[3 * C];
            if (!kRev) {
                // S1^T = Gamma S0^T + (delta U)^T K
                scale_tokens(u, gate + C);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[n][j] *= whole;
            } else {
                // dS0^T = Gamma dS1^T + (s gamma dO)^T Q - (gamma beta E)^T K
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float2 ga = *reinterpret_cast<const float2 *>(gate + n * 8 + tq * 2);
                    const float2 be = *reinterpret_cast<const float2 *>(gate + 2 * C + n * 8 + tq * 2);
                    const float x0 = -ga.x * be.x, x1 = -ga.y * be.y;
                    u[n][0] *= x0; u[n][1] *= x1; u[n][2] *= x0; u[n][3] *= x1;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float4 x = *reinterpret_cast<const float4 *>(hand + (n * 32 + lane) * 16);
                    S[n][0] = fmaf(whole, S[n][0], x.x);
                    S[n][1] = fmaf(whole, S[n][1], x.y);
                    S[n][2] = fmaf(whole, S[n][2], x.z);
                    S[n][3] = fmaf(whole, S[n][3], x.w);
                }
                warp_arrive(hempty(hb));
            }
            add_values_keys<NI, NS, DKP>(u, s + L::K, S);
            warp_arrive(empty1(s1));
        }
        if (!kOut && lane == 0) bulk_wait0();
        float *end = kRev ? p.dh0 : kOut ? p.h_final : nullptr;
        if (end) store_state<NT>(S, end + st_at, v0, p.d_k, p.d_v);
    } else if constexpr (kOut) {
        // ------------------------------------------------ output: O = s gamma Q S0 + (s P) U
        T *out = static_cast<T *>(p.out);
        for (int i = 0; i < n_chunks; ++i) {
            const int s2 = i % N2, hb = i % NH;
            const uint32_t s = base + L::Ring2 + s2 * L::kStage2;
            const float *gate = reinterpret_cast<const float *>(smem + L::Ring2 + s2 * L::kStage2 + L::Gate2);
            const char *hand = smem + L::Hand + (hb * 2 + w) * L::kHand;
            if (!warp_wait(full2(s2), (i / N2) & 1)) break;
            if (!warp_wait(hfull(hb), (i / NH) & 1)) break;
            float o[4][2][4];
            zero<8>(&o[0][0]);
#pragma unroll
            for (int kx = 0; kx < DKP / 16; ++kx) {
                uint4 a[NI];
#pragma unroll
                for (int q = 0; q < NI; ++q)
                    a[q] = *reinterpret_cast<const uint4 *>(hand + ((q * (DKP / 16) + kx) * 32 + lane) * 16);
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int pq = 0; pq < NI; ++pq) {
                        uint32_t f[4];
                        key_a(s + L::Q + pq * C * DKP * 2, m * 16, kx * 16, f);
#pragma unroll
                        for (int pa = 0; pa + pq < NI; ++pa) {
                            ptx::mma16816(o[m][0], f, a[pa].x, a[pa].z);
                            ptx::mma16816(o[m][1], f, a[pa].y, a[pa].w);
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
                uint4 a[NS];
#pragma unroll
                for (int q = 0; q < NS; ++q)
                    a[q] = *reinterpret_cast<const uint4 *>(hand + L::kHandS + ((q * 4 + kx) * 32 + lane) * 16);
#pragma unroll
                for (int m = kx; m < 4; ++m)
#pragma unroll
                    for (int pq = 0; pq < NI; ++pq) {
                        uint32_t f[4];
                        frag_a<128>(s + L::P + pq * kTile * 2, m * 16, kx * 16, f);
#pragma unroll
                        for (int pa = 0; pa + pq < NS; ++pa) {
                            ptx::mma16816(o[m][0], f, a[pa].x, a[pa].z);
                            ptx::mma16816(o[m][1], f, a[pa].y, a[pa].w);
                        }
                    }
            }
            warp_arrive(hempty(hb));
            warp_arrive(empty2(s2));
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = i * C + m * 16 + gr + h * 8;
                    if (r >= len) continue;
                    T *row = out + ((tok0 + r) * p.n_heads + head) * p.d_v;
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int v = v0 + n * 8 + tq * 2;
                        if (v < p.d_v) put2(row + v, o[m][n][h * 2], o[m][n][h * 2 + 1], wide_out, v + 1 < p.d_v);
                    }
                }
        }
    } else if constexpr (kRev) {
        // ------------------------------------------------ G^T = (s gamma dO)^T Q and dO^T P
        for (int i = 0; i < n_chunks; ++i) {
            const int s2 = i % N2, hb = i % NH;
            const uint32_t s = base + L::Ring2 + s2 * L::kStage2;
            const float *gate = reinterpret_cast<const float *>(smem + L::Ring2 + s2 * L::kStage2 + L::Gate2);
            char *hand = smem + L::Hand + (hb * 2 + w) * L::kHand;
            if (!warp_wait(full2(s2), (i / N2) & 1)) break;
            float y[8][4], G[NT][4];
            zero<8>(y);
            zero<NT>(G);
#pragma unroll
            for (int kx = 0; kx < 4; ++kx) {
                uint32_t a[NI][4], d[NS][4];
#pragma unroll
                for (int q = 0; q < NI; ++q) frag_a_t<64>(s + L::dO + q * C * kBlockV * 2, kx * 16, w * 16, a[q]);
#pragma unroll
                for (int n = 0; n <= kx; ++n)
#pragma unroll
                    for (int pb = 0; pb < NS; ++pb) {
                        uint32_t b[4];
                        frag_b_t<128>(s + L::P + pb * kTile * 2, kx * 16, n * 16, b);
#pragma unroll
                        for (int pa = 0; pa < NI && pa + pb < NS; ++pa) {
                            ptx::mma16816(y[2 * n], a[pa], b[0], b[1]);
                            ptx::mma16816(y[2 * n + 1], a[pa], b[2], b[3]);
                        }
                    }
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
#pragma unroll
                for (int n = 0; n < DKP / 16; ++n)
#pragma unroll
                    for (int pb = 0; pb < NI; ++pb) {
                        uint32_t b[4];
                        key_b_t(s + L::Q + pb * C * DKP * 2, kx * 16, n * 16, b);
#pragma unroll
                        for (int pa = 0; pa + pb < NS; ++pa) {
                            ptx::mma16816(G[2 * n], d[pa], b[0], b[1]);
                            ptx::mma16816(G[2 * n + 1], d[pa], b[2], b[3]);
                        }
                    }
            }
            warp_arrive(empty2(s2));
            if (!warp_wait(hempty(hb), ((i / NH) & 1) ^ 1)) break;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<float4 *>(hand + (n * 32 + lane) * 16) = make_float4(G[n][0], G[n][1], G[n][2], G[n][3]);
#pragma unroll
            for (int n = 0; n < 8; ++n)
                *reinterpret_cast<float4 *>(hand + L::kHandS + (n * 32 + lane) * 16) =
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
