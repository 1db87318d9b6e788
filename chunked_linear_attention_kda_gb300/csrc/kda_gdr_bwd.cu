// kda_gdr_bwd.cu -- backward pass of the chunked gated delta rule with one decay per head:
// gradients of <dout, out> + <dh_final, h_final>. Notation and the forward's chunk form as
// in kda_gdr_fwd.cu (X, P with the output scale folded in, gamma, delta, Gamma); s the scale.
//
// Per chunk, with the gradient dS1 of its end state:
//   dU = P^T dO + (delta K) dS1,   E = X^T dU,   dV = beta E
//   dS0 = Gamma dS1 + (s gamma Q)^T dO - (gamma beta K)^T E
// and, from S0, dS1, U and E (local to the chunk, e = e^D, lower triangles):
//   B = s e (dO U^T),  F = e (E U^T) below the diagonal
//   dQ = s gamma (dO S0^T) + B K
//   dK = -gamma beta (E S0^T) + delta (U dS1^T) + B^T Q - (beta F + (beta F)^T) K
//   dbeta_r = E_r.V_r - gamma_r k_r.(E S0^T)_r - sum_j F_rj k_r.k_j
//   dg_i = Gamma <S0, dS1> + sum_{r >= i} a_r + sum_{r < i} b_r + sum_{r >= i > j} M_rj
//   a_r = gamma_r (s q_r.(dO S0^T)_r - beta_r k_r.(E S0^T)_r),  b_r = delta_r k_r.(U dS1^T)_r
//   M_rj = B_rj q_r.k_j - beta_r F_rj k_r.k_j;  its double sum is a running sum of row sums
//   minus column sums.
//
// Three launches: the chunk terms (shared with the forward); one launch with the forward
// chain (S0, U of every chunk) and the reverse chain (dS1, E), which do not depend on each
// other; and the local gradients, all chunks side by side, one CTA per (chunk, key head)
// that walks over the value heads sharing the key head and adds their dQ and dK in
// registers (no atomics: the same call gives the same bits).
//
// bf16, two sequences of 8K tokens, 16 key and 32 value heads, d_k = d_v = 128: 1.51 ms, of it the
// terms 0.11, the chains 0.83 (a step is a chain of dependent products, as in the forward; the
// tensor pipe is active for 52 % of it) and the local gradients 0.56 (2.3 GB at 0.61 of a plain
// copy's bandwidth).
#include <cmath>

#include "kda_gdr_chain.h"

namespace kda {
namespace gdr {
namespace {

// the first half of the blocks runs the reverse chains (the longer ones), the second the forward
template <typename T, int DKP, int NS, int PAIRS>
__global__ void __launch_bounds__(kChainThreads)
    gdr_scan_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                    const GdrArgs p, const Images im, float scale) {
    let_next_kernel_start();
    const unsigned n = gridDim.x / 2;
    if (blockIdx.x >= n) chain<T, DKP, NS, Mode::kStates, PAIRS>(tm_q, tm_k, tm_v, p, im, 2, blockIdx.x - n, scale, false);
    else chain<T, DKP, NS, Mode::kReverse, PAIRS>(tm_q, tm_k, tm_do, p, im, 2, blockIdx.x, scale, false);
}

// ---------------------------------------------------------------- local gradients
// With tcgen05 a CTA is eight warps that compute, each 16 tokens x one half of the key channels
// (or of the 64 columns of a pair product), and three that serve them: one thread copies 16 value
// channels of S0, U, dS1 and E at a time (24 KB, as the chains left them), one thread issues their
// products into tensor memory, one warp sums dbeta and dg. A 64-row accumulator takes 16 lanes of
// each warp's 32 and is read as the fragments of mma.sync, so that the pair products B K, B^T Q and
// F K stay on mma.sync with their operands' scaling in registers; q.k and k.k wait in the other
// 16 lanes. A head's pair products are added while the next head's slices are multiplied.
// 16K tokens of 32 heads: 0.56 ms. With B and F in one plane 0.52; all on mma.sync that took 0.95 (25 %
// of issue slots: two warps a scheduler waited for fragments and for each other).
constexpr int kLocalThreads = 256;          // that compute
constexpr int kCols = kLocalThreads / 128;  // column parts: a warp has 16 tokens x 1 / kCols of the columns
// The products with S0, dS1 and U run on tcgen05 where operands have one and two planes; three
// planes want sums from the smallest product up, which mma.sync's registers give.
template <typename T, int NS>
constexpr bool kTensor = InputPlanes<T>::N == 1 && NS == 2;

template <typename T, int DKP, int NS>
struct LocalSmem {
    static constexpr bool TC = kTensor<T, NS>;
    static constexpr int NI = InputPlanes<T>::N;
    static constexpr int kThreads = kLocalThreads + (TC ? 96 : 0);  // a warp issues products, one loads, one sums dg
    // Slices of the value channels. With tcgen05 16 channels and five buffers, as many as fit: a copy
    // takes 2500 cycles to arrive and its buffer is read for 2000, the products of a slice take 750.
    static constexpr int kSl = TC ? 16 : 32, kStages = TC ? 5 : 1;
    static constexpr int kPlane = C * DKP * 2;
    static constexpr int kIn = C * 32 * 2;  // a plane of 32 channels of dO or V
    // a block of 16 value channels as the chains left it: planes of S and U, planes of dS and E
    static constexpr int kState = 16 * DKP * 2, kPl = 16 * (DKP + C) * 2, kBlock = 2 * NS * kPl;  // kPl: a plane
    static constexpr int S = 0, U = kState, dS = kBlock / 2, E = dS + U, kBlocks = kSl / 16 * kBlock;
    // With tcgen05, dO and V have buffers of their own, three of 32 channels, copied with every
    // other slice; else they lie behind the slice's blocks (fp32 V is read in place).
    static constexpr int dO = TC ? 0 : kBlocks, V = dO + NI * kIn;
    static constexpr int kSlice = TC ? kBlocks : V + (NI == 1 ? kIn : 0);
    static constexpr int Vals = kStages * kSlice, kVals = TC ? 2 * kIn : 0;
    static constexpr int kTile = C * C * 2;  // bytes of a plane of B and F
    static constexpr int K = Vals + 3 * kVals, Q = K + NI * kPlane, Pair = Q + NI * kPlane;
    // q.k and k.k: with tcgen05 in tensor memory. B and F: without it over the first slice buffer,
    // once the slices are done.
    static constexpr int B = TC ? Pair : 0, F = B + NS * kTile;
    static_assert(TC || 2 * NS * kTile <= kSlice, "B and F fit a slice buffer");
    // a head's gates are loaded with its first slice, four slices ahead: with two slices a head
    // the sums of the head three before may still be read
    static constexpr int kGates = TC ? 4 : 1;
    static constexpr int Gate = Pair + (TC ? 2 * NS * kTile : 2 * C * C * 4), Red = Gate + kGates * kGateFloats * 4;
    // Red: [kCols][64] row sums of q.x, k.x, k.x, E.V - F k.k and M over the column parts;
    // [4][64] column sums of M over the row blocks; the warps' parts of <S0, dS1>
    static constexpr int kRed = 5 * kCols * C + 4 * C + kLocalThreads / 32;
    static constexpr int Bars = (Red + kRed * 4 + 7) / 8 * 8;
    // a slice buffer full [kStages], K and Q full; with tcgen05 also a slice buffer read
    // [kStages], a head's sums complete, read, and one to drain by; then the tensor memory's address
    static constexpr int kBars = kStages + 1 + (TC ? kStages + 3 : 0);
    static constexpr int kBytes = Bars + 8 * kBars + 16 + 1024;  // the base is rounded up to 1024
    static_assert(kBytes <= 227 * 1024, "fits an SM");
    static_assert(kSlice % 1024 == 0, "tensor copies land on swizzle boundaries");
};

// a row's sum over the column parts
__device__ __forceinline__ float parts(const float *x, int r) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) s += x[i * C + r];
    return s;
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// eight values from NS planes of bf16
template <int NS>
__device__ __forceinline__ void sum_planes(const char *at, int plane, float *x) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll
    for (int q = NS - 1; q >= 0; --q) {
        const uint4 w = *reinterpret_cast<const uint4 *>(at + q * plane);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] += lo_f(v[e]);
            x[2 * e + 1] += hi_f(v[e]);
        }
    }
}

template <typename T, int DKP, int NS>
__global__ void __launch_bounds__(LocalSmem<T, DKP, NS>::kThreads)
    gdr_local_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     const GdrArgs p, const Images im, float scale, bool wide_k, bool wide_v) {
    constexpr int NI = InputPlanes<T>::N;
    using L = LocalSmem<T, DKP, NS>;
    constexpr bool TC = L::TC;
    // columns of tensor memory: dO [S0 U]^T from 0, E [S0 U]^T, U dS1^T (64 tokens use 16 lanes of
    // each warp's 32)
    [[maybe_unused]] constexpr int kOu = DKP, kXk = DKP + C, kEu = kXk + DKP, kXu = 2 * kXk;
    [[maybe_unused]] constexpr uint32_t kPairs = 16u << 16;  // k.k, then q.k, in the other 16 lanes
    constexpr int KC = DKP / kCols, NH = KC / 16;  // a warp's key channels, in steps of 16
    constexpr int PC = C / kCols, NP = PC / 16;              // its columns of the 64 x 64 products
    extern __shared__ __align__(1024) char smem_raw[];
    char *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tq = lane & 3;
    const int wr = warp & 3, wc = warp >> 2;  // token rows 16 wr .., column part wc
    const int64_t slot = blockIdx.x;
    const Chunk ch = find_chunk(p.cu_seqlens, p.n_seq, slot);
    if (ch.len == 0) return;
    const int kh = blockIdx.y, group = p.n_heads / p.n_k_heads;
    const int n_sl = pad_v(p.d_v) / L::kSl;
    const char *ws = static_cast<const char *>(p.workspace);
    [[maybe_unused]] float *pair = reinterpret_cast<float *>(smem + L::Pair);
    float *gate = reinterpret_cast<float *>(smem + L::Gate);  // TC: head hh's at hh % kGates
    float *red = reinterpret_cast<float *>(smem + L::Red);
    float *r_qx = red, *r_kx = r_qx + kCols * C, *r_ku = r_kx + kCols * C, *r_ef = r_ku + kCols * C;
    float *r_m = r_ef + kCols * C, *c_m = r_m + kCols * C, *r_ss = c_m + 4 * C;

    auto meet = [&](int id) {  // of the warps that compute and the one that sums dg
        if constexpr (TC) ptx::named_sync(id, kLocalThreads + 32);
        else __syncthreads();
    };
    // dbeta and dg of a head, by a warp: two tokens a lane, running sums over the chunk
    auto decay_gradients = [&](int hh, const float *gate) {
        const int head = kh * group + hh;
        const float *gam = gate, *del = gate + C, *bet = gate + 2 * C;
        float whole = 0.f;
#pragma unroll
        for (int i = 0; i < kLocalThreads / 32; ++i) whole += r_ss[i];
        whole *= gate[3 * C];
        Two a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            const float kx = parts(r_kx, r);
            if (r < ch.len)
                p.dbeta[(ch.t0 + r) * p.n_heads + head] = parts(r_ef, r) - gam[r] * kx;
            const float cols = (c_m[r] + c_m[C + r]) + (c_m[2 * C + r] + c_m[3 * C + r]);
            a[i] = add({gam[r] * (scale * parts(r_qx, r) - bet[r] * kx), 0.f}, add({parts(r_m, r), 0.f}, {-cols, 0.f}));
            b[i] = {del[r] * parts(r_ku, r), 0.f};
        }
        // inclusive sums over the tokens of a and b; a0, b0 before token 2 lane
        Two ra = add(a[0], a[1]), rb = add(b[0], b[1]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Two x = {__shfl_up_sync(0xffffffffu, ra.hi, o), __shfl_up_sync(0xffffffffu, ra.lo, o)};
            const Two y = {__shfl_up_sync(0xffffffffu, rb.hi, o), __shfl_up_sync(0xffffffffu, rb.lo, o)};
            if (lane >= o) {
                ra = add(x, ra);
                rb = add(y, rb);
            }
        }
        const Two total = {__shfl_sync(0xffffffffu, ra.hi, 31), __shfl_sync(0xffffffffu, ra.lo, 31)};
        Two a0 = {__shfl_up_sync(0xffffffffu, ra.hi, 1), __shfl_up_sync(0xffffffffu, ra.lo, 1)};
        Two b0 = {__shfl_up_sync(0xffffffffu, rb.hi, 1), __shfl_up_sync(0xffffffffu, rb.lo, 1)};
        if (lane == 0) a0 = b0 = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            const Two before = i ? add(a0, a[0]) : a0, sb = i ? add(b0, b[0]) : b0;
            const Two sum = add(add(total, {-before.hi, -before.lo}), add({whole, 0.f}, sb));
            if (r < ch.len) {  // nothing passes a decay of 0: what the sums leave there is rounding
                const int64_t t = (ch.t0 + r) * p.n_heads + head;
                p.dg[t] = p.g[t] < kGFloor ? 0.f : sum.hi + sum.lo;
            }
        }
    };
    // one thread loads: K and Q, then the slices of the value heads, head after head
    auto bar = [&](int i) { return base + L::Bars + 8 * i; };  // a slice buffer's; kStages: K and Q
    auto used = [&](int i) { return bar(L::kStages + 1 + i); };
    [[maybe_unused]] const uint32_t sums_done = bar(2 * L::kStages + 1), sums_read = sums_done + 8, drain = sums_done + 16;
    const bool image = im.has(ch.t0, ch.len, p.n_tok);
    const size_t img_rec = Images::record(NI, DKP, p.d_v, p.n_k_heads, p.n_heads, 2);
    const size_t kb = Images::key_bytes(NI, DKP), vb = Images::value_bytes(NI, p.d_v);
    const char *img = ws + im.offset + (im.all ? slot : (int64_t)ch.seq) * img_rec;
    bool ok = true;
    int issued = 0;
    // the records of a key head's value heads lie one after the other
    const char *rec = ws + scan_offset(p.n_tok, p.n_seq, p.n_heads, NS) +
                      (slot * p.n_heads + kh * group) * scan_bytes(NS, DKP, p.d_v);
    const char *gates_of = ws + (slot * p.n_heads + kh * group) * terms_bytes(NS) + 2 * NS * kTri;
    auto load = [&](int step, int hh, int sl) {  // slice sl of value head hh; step = hh n_sl + sl
        if (!ok) return;
        ++issued;
        const uint32_t s = base + (step % L::kStages) * L::kSlice, m = bar(step % L::kStages);
        const bool values = !TC || (sl & 1) == 0, gates = TC && sl == 0;  // n_sl is even with tcgen05
        ptx::mbar_arrive_tx(m, L::kSlice + (values ? L::kVals : 0) + (gates ? kGateFloats * 4 : 0));
        bulk_load(s, rec + (size_t)step * L::kBlocks, L::kBlocks, m);
        if (gates)
            bulk_load(base + L::Gate + (hh % L::kGates) * kGateFloats * 4, gates_of + hh * terms_bytes(NS),
                      kGateFloats * 4, m);
        if (values) {
            const uint32_t to = TC ? base + L::Vals + ((step >> 1) % 3) * L::kVals : s;
            const int part = TC ? sl >> 1 : sl, head = kh * group + hh;
            if (image) {
                const char *v = img + 2 * p.n_k_heads * kb + (size_t)part * NI * L::kIn;
                bulk_load(to + L::dO, v + (p.n_heads + head) * vb, NI * L::kIn, m);
                if (NI == 1) bulk_load(to + L::V, v + head * vb, L::kIn, m);
            } else {
                ptx::tma_load_3d(to + L::dO, &tm_do, part * 32, head, (int)ch.t0, m);
                if (NI == 1) ptx::tma_load_3d(to + L::V, &tm_v, part * 32, head, (int)ch.t0, m);
            }
        }
    };
    const int loader = TC ? kLocalThreads + 32 : 0;
    if (tid == loader) {
        for (int i = 0; i <= L::kStages; ++i) ptx::mbar_init(bar(i), 1);
        if constexpr (TC) {
            for (int i = 0; i < L::kStages; ++i) ptx::mbar_init(used(i), kLocalThreads / 32 + 1);
            ptx::mbar_init(sums_done, 1);
            ptx::mbar_init(sums_read, kLocalThreads / 32);
            ptx::mbar_init(drain, 1);
        }
        ptx::mbar_init_fence();
    }
    if constexpr (TC)
        if (warp == kLocalThreads / 32) ptx::tmem_alloc(bar(L::kBars), 512);
    wait_for_previous_kernel();
    if (tid == loader) {
        const uint32_t m = bar(L::kStages);
        ptx::mbar_arrive_tx(m, 2 * NI * L::kPlane);
        if (image) {
            bulk_load(base + L::Q, img + kh * kb, NI * L::kPlane, m);
            bulk_load(base + L::K, img + (p.n_k_heads + kh) * kb, NI * L::kPlane, m);
        } else {
#pragma unroll
            for (int h = 0; h < DKP / 64; ++h) {
                ptx::tma_load_3d(base + L::Q + h * kHalf, &tm_q, h * 64, kh, (int)ch.t0, m);
                ptx::tma_load_3d(base + L::K + h * kHalf, &tm_k, h * 64, kh, (int)ch.t0, m);
            }
        }
        load(0, 0, 0);
    }
    if constexpr (TC) ptx::tc_fence_before();
    __syncthreads();
    [[maybe_unused]] uint32_t tmem = 0;
    if constexpr (TC) {
        ptx::tc_fence_after();
        tmem = *reinterpret_cast<const uint32_t *>(smem + L::Bars + 8 * L::kBars);
    }
    if constexpr (TC)
        if (warp == kLocalThreads / 32 + 2) {  // dbeta and dg
            for (int hh = 0; hh < group; ++hh) {
                meet(2);
                decay_gradients(hh, reinterpret_cast<float *>(smem + L::Gate) + (hh % L::kGates) * kGateFloats);
                if (hh + 1 < group) ptx::named_arrive(1, kLocalThreads + 32);
            }
            __syncthreads();  // the end of the others
            return;
        } else if (warp == kLocalThreads / 32 + 1) {  // a thread loads the slices, as buffers become free
            if (tid == loader) {
                const int steps = group * n_sl;
                for (int step = 1, hh = 0, sl = 1; step < steps; ++step, ++sl) {
                    if (sl == n_sl) {
                        sl = 0;
                        ++hh;
                    }
                    // its buffer, and those of dO and V, need the slice five before to be read, the
                    // gates the one four before
                    static_assert(L::kStages == 5 || !TC, "none of them an earlier one alone");
                    const int last = step - (sl == 0 ? 4 : 5);
                    if (step == 2) ok = wait_bar(bar(L::kStages), 0);  // K and Q first: they are waited for
                    if (step >= L::kStages) ok = wait_bar(used(last % L::kStages), (last / L::kStages) & 1);
                    if (!ok) break;
                    load(step, hh, sl);
                }
                if (!ok) {  // nothing may land in shared memory after the block has gone
                    drain_bar(bar(L::kStages), 0);
                    for (int i = max(0, issued - L::kStages); i < issued; ++i) drain_bar(bar(i % L::kStages), (i / L::kStages) & 1);
                }
            }
            __syncwarp();
            __syncthreads();  // the end of the others
            return;
        } else if (warp == kLocalThreads / 32) {
            // a thread issues the products, up to four slices ahead of the warps that read the sums,
            // and those of the next head while they finish the last one's
            if (lane == 0) {
                constexpr uint32_t id_o = ptx::idesc_bf16(64, DKP + C, 0, 1), id_e = ptx::idesc_bf16(64, DKP + C, 1, 1);
                constexpr uint32_t id_u = ptx::idesc_bf16(64, DKP, 1, 1), id_p = ptx::idesc_bf16(64, C, 0, 0);
                const int steps = group * n_sl;
                // q_r.k_j and k_r.k_j, in the columns of dO U^T and E U^T
                ok = wait_bar(bar(L::kStages), 0);
                if (ok) {
#pragma unroll
                    for (int kx = 0; kx < DKP / 16; ++kx) {
                        const uint32_t at = base + (kx >> 2) * kHalf + (kx & 3) * 32;
                        const uint64_t k = ptx::sdesc_sw128(at + L::K, 16, 1024), q = ptx::sdesc_sw128(at + L::Q, 16, 1024);
                        ptx::umma_ss(tmem + kOu, q, k, id_p, kx > 0);
                        ptx::umma_ss(tmem + kEu, k, k, id_p, kx > 0);
                    }
                    ptx::umma_commit(sums_done);
                }
                // operands of the first buffers; the others' are as many 16-byte units further on
                const uint64_t dO0 = ptx::sdesc_sw64(base + L::Vals, 512);
                const uint64_t one0 = ptx::sdesc_sw128(base, 1024, 1024), all0 = ptx::sdesc_sw128(base, 2048, 1024);
                for (int step = 0, hh = 0, sl = 0, b = 0, vb = 0, phase = 0; ok && step < steps; ++step) {
                    ok = wait_bar(bar(b), phase);
                    if (ok && sl == 0) ok = wait_bar(sums_read, hh & 1);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t more = sl > 0;
                    const uint64_t dO = dO0 + (uint32_t)(vb * L::kVals + (sl & 1) * 32) / 16;
                    const uint64_t one = one0 + (uint32_t)(b * L::kSlice) / 16, all = all0 + (uint32_t)(b * L::kSlice) / 16;
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        ptx::umma_ss(tmem, dO, all + (L::S + i * L::kPl) / 16, id_o, more | (i > 0));
#pragma unroll
                        for (int j = 0; i + j < NS; ++j) {
                            const uint32_t acc = more | (i + j > 0);
                            ptx::umma_ss(tmem + kXk, one + (L::E + i * L::kPl) / 16, all + (L::S + j * L::kPl) / 16, id_e, acc);
                            ptx::umma_ss(tmem + kXu, one + (L::U + i * L::kPl) / 16, all + (L::dS + j * L::kPl) / 16, id_u, acc);
                        }
                    }
                    ptx::umma_commit(used(b));
                    if (++b == L::kStages) {
                        b = 0;
                        phase ^= 1;
                    }
                    if (sl & 1) vb = vb == 2 ? 0 : vb + 1;
                    if (++sl == n_sl) {
                        ptx::umma_commit(sums_done);
                        sl = 0;
                        ++hh;
                    }
                }
                if (!ok) {  // nor may a product run on
                    ptx::umma_commit(drain);
                    drain_bar(drain, 0);
                }
            }
            __syncwarp();
            __syncthreads();  // the others have read the last sums
            ptx::tmem_dealloc(tmem, 512);
            return;
        }
    [[maybe_unused]] const uint32_t lanes = tmem + ((uint32_t)(wr * 32) << 16);
    // A failed wait sets the flag and the block goes on with what is there: nothing more is
    // loaded, and every later wait returns at once.
    ok = wait_bar(bar(L::kStages), 0);

    // q_r.k_j and k_r.k_j of rows 16 wr .., columns PC wc .., kept by each thread for itself
    {
        float kk[2 * NP][4], qk[2 * NP][4];
        if constexpr (TC) {
            ok &= wait_bar(sums_done, 0);
            ptx::tc_fence_after();
            ptx::tmem_ld_frag4(lanes + kOu + wc * PC, reinterpret_cast<uint32_t *>(qk[0]));
            ptx::tmem_ld_frag4(lanes + kEu + wc * PC, reinterpret_cast<uint32_t *>(kk[0]));
            ptx::tmem_ld_wait();
            ptx::tc_fence_before();
            warp_arrive(sums_read);
        } else {
#pragma unroll
            for (int n = 0; n < 2 * NP; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) kk[n][i] = qk[n][i] = 0.f;
#pragma unroll 1
            for (int c = 0; c < DKP; c += 16) {
                uint32_t ak[NI][4], aq[NI][4];
#pragma unroll
                for (int q = 0; q < NI; ++q) {
                    key_a(base + L::K + q * L::kPlane, wr * 16, c, ak[q]);
                    key_a(base + L::Q + q * L::kPlane, wr * 16, c, aq[q]);
                }
#pragma unroll
                for (int n = 0; n < NP; ++n)
                    if (NP * wc + n <= wr) {
                        uint32_t b[NI][4];
#pragma unroll
                        for (int q = 0; q < NI; ++q) key_b(base + L::K + q * L::kPlane, wc * PC + n * 16, c, b[q]);
                        product<NI, NI, NI>(&kk[2 * n], ak, b);
                        product<NI, NI, NI>(&qk[2 * n], aq, b);
                    }
            }
        }
        if constexpr (TC) {
            ptx::tmem_st_frag4(lanes + kPairs + wc * PC, reinterpret_cast<const uint32_t *>(kk[0]));
            ptx::tmem_st_frag4(lanes + kPairs + C + wc * PC, reinterpret_cast<const uint32_t *>(qk[0]));
            ptx::tmem_st_wait();
        } else {
#pragma unroll
            for (int n = 0; n < 2 * NP; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    pair[(n * 4 + i) * kLocalThreads + tid] = kk[n][i];
                    pair[(8 * NP + n * 4 + i) * kLocalThreads + tid] = qk[n][i];
                }
        }
    }

    float dq[2 * NH][4], dk[2 * NH][4];  // this warp's rows and key channels
#pragma unroll
    for (int n = 0; n < 2 * NH; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) dq[n][i] = dk[n][i] = 0.f;

    // dQ += B K, dK += B^T Q - (beta F + its transpose) K
    auto add_pairs = [&]() {
#pragma unroll
        for (int kx = 0; kx < 4; ++kx) {
            uint32_t ab[NS][4], at[NS][4], af[NS][4];
#pragma unroll
            for (int q = 0; q < NS; ++q) {
                frag_a<128>(base + L::B + q * L::kTile, wr * 16, kx * 16, ab[q]);
                frag_a_t<128>(base + L::B + q * L::kTile, kx * 16, wr * 16, at[q]);
                frag_a<128>(base + L::F + q * L::kTile, wr * 16, kx * 16, af[q]);
                uint32_t ft[4];
                frag_a_t<128>(base + L::F + q * L::kTile, kx * 16, wr * 16, ft);
#pragma unroll
                for (int i = 0; i < 4; ++i) af[q][i] |= ft[i];  // of the two at least one is +0
            }
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                uint32_t b[NI][4];
#pragma unroll
                for (int q = 0; q < NI; ++q) key_b_t(base + L::K + q * L::kPlane, kx * 16, wc * KC + n * 16, b[q]);
                if (kx <= wr) product<NS, NI, NS>(&dq[2 * n], ab, b);
                product<NS, NI, NS>(&dk[2 * n], af, b);
                if (kx < wr) continue;  // B is lower triangular
#pragma unroll
                for (int q = 0; q < NI; ++q) key_b_t(base + L::Q + q * L::kPlane, kx * 16, wc * KC + n * 16, b[q]);
                product<NS, NI, NS>(&dk[2 * n], at, b);
            }
        }
    };

    for (int hh = 0; hh < group; ++hh) {
        const int head = kh * group + hh;
        constexpr int XT = TC ? 4 : 2 * NH;  // tiles of 8 key channels in registers at a time
        float xq[XT][4], xk[XT][4], xu[XT][4], ou[2 * NP][4], eu[2 * NP][4];
        if constexpr (!TC) {
            zero<XT>(xq);
            zero<XT>(xk);
            zero<XT>(xu);
            zero<2 * NP>(ou);
            zero<2 * NP>(eu);
        }
        float ev[2] = {0.f, 0.f}, ss = 0.f;
        if constexpr (TC) {
            gate = reinterpret_cast<float *>(smem + L::Gate) + (hh % L::kGates) * kGateFloats;
        } else {
            for (int i = tid; i < kGateFloats; i += kLocalThreads)
                gate[i] = reinterpret_cast<const float *>(ws + (slot * p.n_heads + head) * terms_bytes(NS) + 2 * NS * kTri)[i];
        }

        for (int sl = 0; sl < n_sl; ++sl) {
            const int step = hh * n_sl + sl;
            if (!TC && tid == 0 && step > 0) load(step, hh, sl);
            ok &= wait_bar(bar(step % L::kStages), (step / L::kStages) & 1);
            if (!TC && sl == 0) __syncthreads();  // the gates
            const uint32_t s = base + (step % L::kStages) * L::kSlice;
            // with tcgen05 the column parts take turns, a slice each; else the first sums, the second writes dV
            const bool sums = wc == (TC ? sl & 1 : 0), writes = wc == (TC ? sl & 1 : 1);
            if (sums)  // <S0, dS1>: both lie in the same order
#pragma unroll
                for (int i = 0; i < L::kSl / 16 * L::kState; i += 128 * 16) {
                    const char *at = smem + (s - base) + i / L::kState * L::kBlock + i % L::kState + (tid & 127) * 16;
                    float x[8], y[8];
                    sum_planes<NS>(at + L::S, L::kPl, x);
                    sum_planes<NS>(at + L::dS, L::kPl, y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], y[e], ss);
                }
#pragma unroll
            for (int kx = 0; kx < L::kSl / 16; ++kx) {  // 16 value channels
                const int vx = TC ? sl & 1 : kx;         // of the 32 that dO and V are copied by
                if (TC && !sums) break;
                uint32_t ae[NS][4];
#pragma unroll
                for (int q = 0; q < NS; ++q) frag_a_t<128>(s + kx * L::kBlock + L::E + q * L::kPl, 0, wr * 16, ae[q]);
                if (sums) {  // E_r.V_r
                    uint32_t av[4];
                    if constexpr (NI == 1) frag_a<64>((TC ? base + L::Vals + ((step >> 1) % 3) * L::kVals : s) + L::V, wr * 16, vx * 16, av);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x0 = 0.f, x1 = 0.f, z0 = 0.f, z1 = 0.f;
#pragma unroll
                        for (int q = 0; q < NS; ++q) { x0 += lo_f(ae[q][i]); x1 += hi_f(ae[q][i]); }
                        if constexpr (NI == 1) {
                            z0 = lo_f(av[i]);
                            z1 = hi_f(av[i]);
                        } else {
                            const int r = wr * 16 + gr + (i & 1) * 8, v = sl * L::kSl + kx * 16 + (i >> 1) * 8 + tq * 2;
                            const float *at = static_cast<const float *>(p.v) + (ch.t0 + r) * p.v_stride + (int64_t)head * p.d_v + v;
                            if (r < ch.len && v < p.d_v) z0 = at[0];
                            if (r < ch.len && v + 1 < p.d_v) z1 = at[1];
                        }
                        ev[i & 1] = fmaf(x0, z0, fmaf(x1, z1, ev[i & 1]));
                    }
                }
                if (writes) {  // dV = beta E
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x0 = 0.f, x1 = 0.f;
#pragma unroll
                        for (int q = 0; q < NS; ++q) { x0 += lo_f(ae[q][i]); x1 += hi_f(ae[q][i]); }
                        const int r = wr * 16 + gr + (i & 1) * 8, v = sl * L::kSl + kx * 16 + (i >> 1) * 8 + tq * 2;
                        if (r < ch.len && v < p.d_v) {
                            const float be = gate[2 * C + r];
                            put2(static_cast<T *>(p.dv) + ((ch.t0 + r) * p.n_heads + head) * p.d_v + v, be * x0, be * x1,
                                 wide_v, v + 1 < p.d_v);
                        }
                    }
                }
                if constexpr (!TC) {
                    uint32_t ao[NI][4], au[NS][4];
#pragma unroll
                    for (int q = 0; q < NI; ++q) frag_a<64>(s + L::dO + q * L::kIn, wr * 16, kx * 16, ao[q]);
#pragma unroll
                    for (int q = 0; q < NS; ++q) frag_a_t<128>(s + kx * L::kBlock + L::U + q * L::kPl, 0, wr * 16, au[q]);
                    // dO S0^T, E S0^T, U dS1^T
#pragma unroll
                    for (int n = 0; n < NH; ++n) {
                        const int c = wc * KC + n * 16;
                        const uint32_t at = s + kx * L::kBlock + state_half(c);
                        uint32_t b[NS][4];
#pragma unroll
                        for (int q = 0; q < NS; ++q) frag_b_t<128>(at + L::S + q * L::kPl, 0, c & 63, b[q]);
                        product<NI, NS, NS>(&xq[2 * n], ao, b);
                        product<NS, NS, NS>(&xk[2 * n], ae, b);
#pragma unroll
                        for (int q = 0; q < NS; ++q) frag_b_t<128>(at + L::dS + q * L::kPl, 0, c & 63, b[q]);
                        product<NS, NS, NS>(&xu[2 * n], au, b);
                    }
                    // dO U^T, E U^T
#pragma unroll
                    for (int n = 0; n < NP; ++n)
                        if (NP * wc + n <= wr) {
                            uint32_t b[NS][4];
#pragma unroll
                            for (int q = 0; q < NS; ++q) frag_b_t<128>(s + kx * L::kBlock + L::U + q * L::kPl, 0, wc * PC + n * 16, b[q]);
                            product<NI, NS, NS>(&ou[2 * n], ao, b);
                            product<NS, NS, NS>(&eu[2 * n], ae, b);
                        }
                }
            }
            if constexpr (TC) warp_arrive(used(step % L::kStages));
            else __syncthreads();
        }
        if constexpr (TC) {
            if (hh > 0) add_pairs();  // the last head's
            ok &= wait_bar(sums_done, (hh + 1) & 1);
            ptx::tc_fence_after();
            if (hh > 0) meet(1);  // B, F and the sums of the head before are done with
        }

        // row dots with q and k, and the products scaled into the head sums
        const float *gam = gate, *del = gate + C, *bet = gate + 2 * C;
        const float2 *G2 = reinterpret_cast<const float2 *>(gate + 4 * C);
        {
            float qx[2] = {0.f, 0.f}, kx_[2] = {0.f, 0.f}, ku[2] = {0.f, 0.f};
#pragma unroll
            for (int part = 0; part < 2 * NH / XT; ++part) {
                if constexpr (TC) {
                    const uint32_t at = lanes + wc * KC + part * 32;
                    ptx::tmem_ld_frag4(at, reinterpret_cast<uint32_t *>(xq[0]));
                    ptx::tmem_ld_frag4(at + kXk, reinterpret_cast<uint32_t *>(xk[0]));
                    ptx::tmem_ld_frag4(at + kXu, reinterpret_cast<uint32_t *>(xu[0]));
                    ptx::tmem_ld_wait();
                }
#pragma unroll
                for (int n = 0; n < XT; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = wr * 16 + gr + 8 * h, t = part * XT + n;
                        const uint32_t at = key_off(r, wc * KC + t * 8 + tq * 2);
                        float k0 = 0.f, k1 = 0.f, q0 = 0.f, q1 = 0.f;
#pragma unroll
                        for (int q = 0; q < NI; ++q) {
                            const uint32_t wk = *reinterpret_cast<const uint32_t *>(smem + L::K + q * L::kPlane + at);
                            const uint32_t wq = *reinterpret_cast<const uint32_t *>(smem + L::Q + q * L::kPlane + at);
                            k0 += lo_f(wk); k1 += hi_f(wk); q0 += lo_f(wq); q1 += hi_f(wq);
                        }
                        qx[h] = fmaf(q0, xq[n][2 * h], fmaf(q1, xq[n][2 * h + 1], qx[h]));
                        kx_[h] = fmaf(k0, xk[n][2 * h], fmaf(k1, xk[n][2 * h + 1], kx_[h]));
                        ku[h] = fmaf(k0, xu[n][2 * h], fmaf(k1, xu[n][2 * h + 1], ku[h]));
                        const float sg = scale * gam[r], gb = -gam[r] * bet[r], de = del[r];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            dq[t][2 * h + i] = fmaf(sg, xq[n][2 * h + i], dq[t][2 * h + i]);
                            dk[t][2 * h + i] = fmaf(gb, xk[n][2 * h + i], fmaf(de, xu[n][2 * h + i], dk[t][2 * h + i]));
                        }
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = wr * 16 + gr + 8 * h;
                const float a = quad_sum(qx[h]), b = quad_sum(kx_[h]), d = quad_sum(ku[h]);
                if (tq == 0) {
                    r_qx[wc * C + r] = a;
                    r_kx[wc * C + r] = b;
                    r_ku[wc * C + r] = d;
                }
            }
        }
        float kp[2 * NP][4], qp[2 * NP][4];  // k.k and q.k
        // B (lower) and -beta F (below the diagonal) as operands; row and column sums
        if constexpr (TC) {
            ptx::tmem_ld_frag4(lanes + kOu + wc * PC, reinterpret_cast<uint32_t *>(ou[0]));
            ptx::tmem_ld_frag4(lanes + kEu + wc * PC, reinterpret_cast<uint32_t *>(eu[0]));
            ptx::tmem_ld_wait();
            ptx::tc_fence_before();
            warp_arrive(sums_read);
            ptx::tmem_ld_frag4(lanes + kPairs + wc * PC, reinterpret_cast<uint32_t *>(kp[0]));
            ptx::tmem_ld_frag4(lanes + kPairs + C + wc * PC, reinterpret_cast<uint32_t *>(qp[0]));
            ptx::tmem_ld_wait();
        }
        {
            float fk[2] = {0.f, 0.f}, mr[2] = {0.f, 0.f};
#pragma unroll
            for (int n = 0; n < 2 * NP; ++n) {
                float mc[2] = {0.f, 0.f};
                const int j = wc * PC + n * 8 + tq * 2;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = wr * 16 + gr + 8 * h;
                    float bv[2], fv[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float kk = TC ? kp[n][2 * h + i] : pair[(n * 4 + 2 * h + i) * kLocalThreads + tid];
                        const float qk = TC ? qp[n][2 * h + i] : pair[(8 * NP + n * 4 + 2 * h + i) * kLocalThreads + tid];
                        const float d = (G2[r].x - G2[j + i].x) + (G2[r].y - G2[j + i].y);
                        const float e = j + i <= r ? ex2(d) : 0.f;
                        bv[i] = j + i <= r ? scale * e * ou[n][2 * h + i] : 0.f;
                        const float f = j + i < r ? e * eu[n][2 * h + i] : 0.f;
                        fv[i] = j + i < r ? -bet[r] * f : 0.f;
                        fk[h] = fmaf(f, kk, fk[h]);
                        const float m = j + i < r ? fmaf(bv[i], qk, fv[i] * kk) : 0.f;
                        mr[h] += m;
                        mc[i] += m;
                    }
                    uint32_t wb[NS], wf[NS];
                    split2<NS>(bv[0], bv[1], wb);
                    split2<NS>(fv[0], fv[1], wf);
#pragma unroll
                    for (int q = 0; q < NS; ++q) {
                        *reinterpret_cast<uint32_t *>(smem + L::B + q * L::kTile + tile_off<128>(r, j)) = wb[q];
                        *reinterpret_cast<uint32_t *>(smem + L::F + q * L::kTile + tile_off<128>(r, j)) = wf[q];
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mc[i] += __shfl_xor_sync(0xffffffffu, mc[i], o);
                    if (gr == 0) c_m[wr * C + j + i] = mc[i];
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float a = quad_sum(ev[h] - fk[h]), b = quad_sum(mr[h]);
                if (tq == 0) {
                    r_ef[wc * C + wr * 16 + gr + 8 * h] = a;
                    r_m[wc * C + wr * 16 + gr + 8 * h] = b;
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (lane == 0) r_ss[warp] = ss;
        }
        meet(2);
        if (!TC && warp == 0) decay_gradients(hh, gate);
        // With tcgen05 the next head's slices come first: their buffers are waited for.
        if (!TC || hh + 1 == group) add_pairs();
        if constexpr (!TC) {
            ptx::fence_proxy_async();  // B and F were written by plain stores; the next copies overwrite them
            __syncthreads();           // B, F, the gates and the sums are done with
        }
    }
    if (!TC && !ok && tid == 0) {  // nothing may land in shared memory after the block has gone
        drain_bar(bar(L::kStages), 0);
        for (int i = max(0, issued - L::kStages); i < issued; ++i) drain_bar(bar(i % L::kStages), (i / L::kStages) & 1);
    }
    if constexpr (TC) {
        ptx::tc_fence_before();
        __syncthreads();  // the tensor memory may be freed
    }
    // write the key head's gradients
#pragma unroll
    for (int n = 0; n < 2 * NH; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = wr * 16 + gr + 8 * h, c = wc * KC + n * 8 + tq * 2;
            if (r < ch.len && c < p.d_k) {
                const size_t at = ((ch.t0 + r) * p.n_k_heads + kh) * p.d_k + c;
                put2(static_cast<T *>(p.dq) + at, dq[n][2 * h], dq[n][2 * h + 1], wide_k, c + 1 < p.d_k);
                put2(static_cast<T *>(p.dk) + at, dk[n][2 * h], dk[n][2 * h + 1], wide_k, c + 1 < p.d_k);
            }
        }
}

template <typename T, int DKP, int NS>
cudaError_t backward(const GdrArgs &p, cudaStream_t stream) {
    constexpr int NI = InputPlanes<T>::N;
    const float scale = 1.f / std::sqrt((float)p.d_k);
    ChainMaps maps;
    const Images im{!maps.make<T>(p, true), scan_offset(p.n_tok, p.n_seq, p.n_heads, NS) +
                                                (size_t)n_slots(p.n_tok, p.n_seq) * p.n_heads * scan_bytes(NS, DKP, p.d_v)};
    cudaError_t e = launch_gdr_terms(p, im, 2, NS, stream);
    if (e != cudaSuccess) return e;
    auto scan = [&](auto kernel, int pairs, int fwd, int rev) {
        return launch_dependent(kernel, 2 * chain_blocks(p, pairs), kChainThreads, fwd > rev ? fwd : rev, stream, maps.q,
                                maps.k, maps.v, maps.dout, p, im, scale);
    };
    bool wide_scan = false;
    if constexpr (NS == 2) wide_scan = scan_pairs(p) == 4;
    if constexpr (NS == 2)
        if (wide_scan)
            e = scan(gdr_scan_kernel<T, DKP, NS, 4>, 4, ChainSmem<NI, DKP, NS, Mode::kStates, 4>::kBytes,
                     ChainSmem<NI, DKP, NS, Mode::kReverse, 4>::kBytes);
    if (!wide_scan)
        e = scan(gdr_scan_kernel<T, DKP, NS, 2>, 2, ChainSmem<NI, DKP, NS, Mode::kStates, 2>::kBytes,
                 ChainSmem<NI, DKP, NS, Mode::kReverse, 2>::kBytes);
    if (e != cudaSuccess || p.n_tok == 0) return e;
    auto wide = [](const void *x, int d) { return d % 2 == 0 && ((uintptr_t)x % (2 * sizeof(T))) == 0; };
    return launch_dependent(gdr_local_kernel<T, DKP, NS>, dim3((unsigned)n_slots(p.n_tok, p.n_seq), p.n_k_heads),
                            LocalSmem<T, DKP, NS>::kThreads, LocalSmem<T, DKP, NS>::kBytes, stream, maps.q, maps.k, maps.v, maps.dout, p, im,
                            scale, wide(p.dq, p.d_k) && wide(p.dk, p.d_k), wide(p.dv, p.d_v));
}

// Planes of the intermediates. dg sums inner products of states with state gradients, which
// cancel. Over 110 bf16 problems of 1 to 32 heads and 4 to 2900 tokens its error with two planes
// is up to 1.2e-5 of its norm below 2000 (token, head) pairs, up to 7.2e-6 from there to 8192 and
// beyond; with three it stays at 4.2e-7. Three planes take about twice the time: 78 against 43 us
// at 2048 pairs, 281 against 142 us at 32768, 3.53 against 1.51 ms at 524288. Calls whose norm few
// sums make up take three, up to four times the size below which the error is largest: those are short
// calls. The rule sees the call alone (a sequence's length is on the device), so a sequence's
// gradients have the accuracy of the call that it is packed into.
int planes(int64_t n_tok, int32_t n_heads, bool bf16) {
    return bf16 && n_tok * n_heads >= 8192 ? 2 : 3;
}

}  // namespace
}  // namespace gdr

size_t gdr_bwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k,
                               int32_t d_v, bool bf16) {
    const int ns = gdr::planes(n_tok, n_heads, bf16), dkp = d_k <= 64 ? 64 : 128;
    return gdr::scan_offset(n_tok, n_seq, n_heads, ns) +
           (size_t)gdr::n_slots(n_tok, n_seq) * (n_heads * gdr::scan_bytes(ns, dkp, d_v) +
                                                 gdr::Images::record(bf16 ? 1 : 3, dkp, d_v, n_k_heads, n_heads, 2));
}

cudaError_t launch_gdr_bwd(const GdrArgs &p, cudaStream_t stream) {
    using bf16 = __nv_bfloat16;
    if (!p.bf16) return p.d_k <= 64 ? gdr::backward<float, 64, 3>(p, stream) : gdr::backward<float, 128, 3>(p, stream);
    if (gdr::planes(p.n_tok, p.n_heads, true) == 3)
        return p.d_k <= 64 ? gdr::backward<bf16, 64, 3>(p, stream) : gdr::backward<bf16, 128, 3>(p, stream);
    return p.d_k <= 64 ? gdr::backward<bf16, 64, 2>(p, stream) : gdr::backward<bf16, 128, 2>(p, stream);
}

cudaError_t read_gdr_bwd_flags(unsigned int *flags, bool reset, cudaStream_t stream) {
    return gdr::read_flags(flags, reset, stream);
}

}  // namespace kda
