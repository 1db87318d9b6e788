// kda_dla_fwd.cu -- chunked forward of linear attention with one decay per head, bf16 inputs, on
// tcgen05; the formulas are in kda_dla.h.
//
// A CTA walks over a segment of one sequence and head in tiles of 64 tokens and carries the state
// S^T (d_v x d_k, fp32, in the registers of eight warps). Per tile, with tokens as columns so that
// every product has 128 rows:
//   Q K^T                        64 x 64, both tiles as they were copied
//   O1 = S^T Q^T                 S^T as two bf16 planes in tensor memory (the A operand)
//   O2 = V^T P^T                 P = e Q K^T as two planes in shared memory
//   dS^T = V^T K'                K' = delta K as two planes in shared memory
//   o = scale (gamma O1 + O2),  S^T <- Gamma S^T + dS^T
// The state is converted once a tile, off the products' path: what waits for it is O1 alone.
//
// A long sequence is cut into segments, so that few heads fill the GPU: a first launch forms what
// each segment adds to the state (kda_dla_states.h: K and V are read once more), a second one the
// states at the segments' starts, a third the output, all segments side by side.
#include <cmath>

#include "kda_dla_states.h"

namespace kda {
namespace dla {
namespace {

// warps: 0 issues products, 1 forms gates, 2 and 3 load, 4..7 K' and P, 8..15 the state, 16..19 the output
constexpr int kFwdThreads = 640;

template <int DK>
struct FwdSmem {
    static constexpr int kKey = DK / 64 * kHalf, kVal = 2 * kHalf;
    static constexpr int Q = 0, K = kKey, V = 2 * kKey, kStage = V + kVal;
    static constexpr int kStages = 3;
    static constexpr int Kp = kStages * kStage, P = Kp + 2 * kKey, O = P + 2 * kHalf, Gate = O + 2 * kHalf;
    static constexpr int kGates = 4;
    static constexpr int Ring = Gate + kGates * (int)sizeof(TileGates), Bars = Ring + kAhead * C * 4;
    // full, empty [stages], gates full, empty [4], QK full, empty [2], then one each
    static constexpr int Full = 0, Empty = kStages, GFull = 2 * kStages, GEmpty = GFull + kGates, QkFull = GEmpty + kGates,
                         QkEmpty = QkFull + 2, PFull = QkEmpty + 2, PEmpty = PFull + 1, KpFull = PEmpty + 1,
                         KpEmpty = KpFull + 1, DsFull = KpEmpty + 1, DsEmpty = DsFull + 1, SFull = DsEmpty + 1,
                         SEmpty = SFull + 1, O1Empty = SEmpty + 1, O2Full = O1Empty + 1, O2Empty = O2Full + 1, Drain = O2Empty + 1,
                         kBars = Drain + 1;
    static constexpr int kBytes = Bars + 8 * kBars + 16 + 1024;  // the base is rounded up to 1024
    static_assert(kBytes <= 227 * 1024, "fits an SM");
};
// columns of tensor memory
constexpr int kTmDs = 0, kTmS = 128, kTmO1 = 256, kTmO2 = 320, kTmQk = 384;

template <int DK>
__global__ void __launch_bounds__(kFwdThreads, 1)
    dla_forward_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const DlaArgs p, const Plan plan, bool copies,
                       bool wide_out) {
    using L = FwdSmem<DK>;
    constexpr int S = L::kStages;
    extern __shared__ __align__(1024) char smem_raw[];
    char *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int head = blockIdx.x % p.n_heads, kh = head / (p.n_heads / p.n_k_heads);
    const int64_t slot = blockIdx.x / p.n_heads;
    const Segment sg = find_segment(p.cu_seqlens, p.n_seq, slot, plan.seg);
    const int64_t state_at = ((int64_t)sg.seq * p.n_heads + head) * p.d_k * p.d_v;
    if (sg.len == 0) {
        if (sg.last && p.h_final)  // an empty sequence
            for (int i = tid; i < p.d_k * p.d_v; i += kFwdThreads) p.h_final[state_at + i] = p.h0 ? p.h0[state_at + i] : 0.f;
        return;
    }
    const int nc = (int)((sg.len + C - 1) / C);
    const bool keep_end = sg.last && p.h_final;  // else the last tile adds to no state
    auto bar = [&](int i) { return base + L::Bars + 8 * i; };
    auto gate = [&](int c) { return reinterpret_cast<TileGates *>(smem + L::Gate) + c % L::kGates; };
    auto rows_of = [&](int c) { return (int)min((int64_t)C, sg.len - (int64_t)c * C); };

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            ptx::mbar_init(bar(L::Full + i), 1);
            ptx::mbar_init(bar(L::Empty + i), 1 + 4);
        }
        for (int i = 0; i < L::kGates; ++i) {
            ptx::mbar_init(bar(L::GFull + i), 1);
            ptx::mbar_init(bar(L::GEmpty + i), 4 + 8 + 4);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(L::QkFull + i), 1);
            ptx::mbar_init(bar(L::QkEmpty + i), 4);
        }
        ptx::mbar_init(bar(L::PFull), 4);
        ptx::mbar_init(bar(L::PEmpty), 1);
        ptx::mbar_init(bar(L::KpFull), 4);
        ptx::mbar_init(bar(L::KpEmpty), 1);
        ptx::mbar_init(bar(L::DsFull), 1);
        ptx::mbar_init(bar(L::DsEmpty), 8);
        ptx::mbar_init(bar(L::SFull), 8);
        ptx::mbar_init(bar(L::SEmpty), 1);
        ptx::mbar_init(bar(L::O1Empty), 4);
        ptx::mbar_init(bar(L::O2Full), 1);
        ptx::mbar_init(bar(L::O2Empty), 4);
        ptx::mbar_init(bar(L::Drain), 1);
        ptx::mbar_init_fence();
    }
    if (warp == 0) ptx::tmem_alloc(bar(L::kBars), 512);
    // P is zero above its diagonal blocks, V in channels that no value head has
    for (int i = tid; i < 2 * kHalf / 16; i += kFwdThreads) reinterpret_cast<uint4 *>(smem + L::P)[i] = make_uint4(0, 0, 0, 0);
    if (p.d_v <= 64)
        for (int i = tid; i < S * kHalf / 16; i += kFwdThreads)
            *reinterpret_cast<uint4 *>(smem + (i / (kHalf / 16)) * L::kStage + L::V + kHalf + (i % (kHalf / 16)) * 16) = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<const uint32_t *>(smem + L::Bars + 8 * L::kBars);
    bool ok = true;
    // A failed wait sets the flag: every later one returns at once, nothing more is loaded, and the
    // block ends with what is there.
    auto wait = [&](int b, int parity) { ok = wait_bar(bar(b), parity & 1) && ok; };

    if (warp == 0) {
        // The whole warp walks, one lane issues: operands by offsets in uniform registers.
        constexpr uint32_t id_qk = ptx::idesc_bf16(64, C, 0, 0), id_o1 = ptx::idesc_bf16(128, C, 0, 0);
        constexpr uint32_t id_o2 = ptx::idesc_bf16(128, C, 1, 0), id_ds = ptx::idesc_bf16(128, DK, 1, 1);
        const uint32_t leader = ptx::elect_one();
        const uint64_t q0 = ptx::sdesc_sw128(base + L::Q, 16, 1024), k0 = ptx::sdesc_sw128(base + L::K, 16, 1024);
        const uint64_t v0 = ptx::sdesc_sw128(base + L::V, kHalf, 1024), kp = ptx::sdesc_sw128(base + L::Kp, kHalf, 1024);
        const uint64_t pp = ptx::sdesc_sw128(base + L::P, 16, 1024);
        auto step = [](int k) { return (uint32_t)((k >> 2) * kHalf + (k & 3) * 32) / 16; };  // 16 channels, K-major
        int next = 0, next_phase = 0;  // the stage of the next Q K^T
        auto pairs = [&](int c) {
            wait(L::Full + next, next_phase);
            if (c >= 2) wait(L::QkEmpty + (c & 1), (c >> 1) - 1);
            ptx::tc_fence_after();
            const uint32_t at = (uint32_t)next * (L::kStage / 16);
#pragma unroll
            for (int k = 0; k < DK / 16; ++k)
                ptx::umma_ss_by(leader, tmem + kTmQk + (c & 1) * C, q0 + (at + step(k)), k0 + (at + step(k)), id_qk, k > 0);
            ptx::umma_commit_by(leader, bar(L::QkFull + (c & 1)));
            if (++next == S) {
                next = 0;
                next_phase ^= 1;
            }
        };
        pairs(0);
        int s = 0;
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
            // in the order in which their operands come: dS^T is waited for by the state's warps while
            // O1 is formed, and O1 by the next tile's planes of S
            if (c + 1 < nc) pairs(c + 1);
            const uint32_t at = (uint32_t)s * (L::kStage / 16);
            if (c + 1 < nc || keep_end) {
                wait(L::KpFull, c);
                if (c > 0) wait(L::DsEmpty, c - 1);
                ptx::tc_fence_after();
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int k = 0; k < C / 16; ++k)
                        ptx::umma_ss_by(leader, tmem + kTmDs, v0 + (at + 128 * k), kp + (i * L::kKey / 16 + 128 * k), id_ds, i + k > 0);
                ptx::umma_commit_by(leader, bar(L::DsFull));
                ptx::umma_commit_by(leader, bar(L::KpEmpty));
            }
            wait(L::SFull, c);
            if (c > 0) wait(L::O1Empty, c - 1);
            ptx::tc_fence_after();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
                    ptx::umma_ts_by(leader, tmem + kTmO1, tmem + kTmS + i * (DK / 2) + 8 * k, q0 + (at + step(k)), id_o1, i + k > 0);
            ptx::umma_commit_by(leader, bar(L::SEmpty));
            wait(L::PFull, c);
            if (c > 0) wait(L::O2Empty, c - 1);
            ptx::tc_fence_after();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < C / 16; ++k)
                    ptx::umma_ss_by(leader, tmem + kTmO2, v0 + (at + 128 * k), pp + (i * kHalf + k * 32) / 16, id_o2, i + k > 0);
            ptx::umma_commit_by(leader, bar(L::O2Full));
            ptx::umma_commit_by(leader, bar(L::PEmpty));
            ptx::umma_commit_by(leader, bar(L::Empty + s));
            if (++s == S) s = 0;
        }
        ptx::umma_commit_by(leader, bar(L::Drain));
        drain_bar(bar(L::Drain), 0);
    } else if (warp == 1) {
        walk_gates<false>(
            p, reinterpret_cast<float *>(smem + L::Ring), sg.t0, head, nc, [](int n) { return n; }, rows_of, gate,
            [&](int n) { if (n >= L::kGates) wait(L::GEmpty + n % L::kGates, n / L::kGates - 1); },
            [&](int n) { warp_arrive(bar(L::GFull + n % L::kGates)); });
    } else if (warp < 4) {
        const Source q{&tm_q, static_cast<const __nv_bfloat16 *>(p.q), p.q_stride, kh, p.d_k, DK / 64, plan.vec_q};
        const Source k{&tm_k, static_cast<const __nv_bfloat16 *>(p.k), p.k_stride, kh, p.d_k, DK / 64, plan.vec_k};
        const Source v{&tm_v, static_cast<const __nv_bfloat16 *>(p.v), p.v_stride, head, p.d_v, p.d_v > 64 ? 2 : 1, plan.vec_v};
        int copied = 0;  // tiles whose copies were begun
        for (int c = 0; c < nc; ++c) {
            const int s = c % S, rows = rows_of(c);
            if (c >= S) wait(L::Empty + s, c / S - 1);
            ok = __all_sync(0xffffffffu, ok);
            const uint32_t at = base + s * L::kStage;
            const int64_t t0 = sg.t0 + (int64_t)c * C;
            if (copies && rows == C) {
                if (ok && warp == 2 && lane == 0) {
                    const uint32_t m = bar(L::Full + s);
                    ptx::mbar_arrive_tx(m, 2 * L::kKey + v.halves * kHalf);
                    tile_by_copy(k, at + L::K, t0, m);
                    tile_by_copy(q, at + L::Q, t0, m);
                    tile_by_copy(v, at + L::V, t0, m);
                    copied = c + 1;
                }
            } else {
                if (ok) {
                    tile_by_threads(k, at + L::K, t0, rows, tid - 64, 64);
                    tile_by_threads(q, at + L::Q, t0, rows, tid - 64, 64);
                    tile_by_threads(v, at + L::V, t0, rows, tid - 64, 64);
                }
                tile_loaded(bar(L::Full + s));
            }
        }
        // nothing may land in shared memory after the block has gone
        if (!ok)
            for (int c = max(0, copied - S); c < copied; ++c) drain_bar(bar(L::Full + c % S), (c / S) & 1);
    } else if (warp < 8) {
        const int w = warp - 4, gr = lane >> 2, tq = lane & 3;
        const uint32_t lanes = tmem + ((uint32_t)(w * 32) << 16);
        const uint32_t put_at = base + L::P, row = 16 * w + ((lane >> 3) & 1) * 8 + (lane & 7), col8 = (lane >> 4) * 8;
        auto keys = [&](int c) {  // K' of tile c
            const int s = c % S;
            wait(L::GFull + c % L::kGates, c / L::kGates);
            wait(L::Full + s, c / S);
            if (c > 0) wait(L::KpEmpty, c - 1);
            scale_rows(smem + s * L::kStage + L::K, smem + L::Kp, L::kKey, *gate(c), L::kKey, tid - 128, 128);
            ptx::fence_proxy_async();
            warp_arrive(bar(L::KpFull));
            warp_arrive(bar(L::Empty + s));
        };
        keys(0);
        for (int c = 0; c < nc; ++c) {
            const TileGates &g = *gate(c);
            wait(L::QkFull + (c & 1), c >> 1);
            ptx::tc_fence_after();
            const int r0 = 16 * w + gr;
            const float2 G0 = g.G[r0], G1 = g.G[r0 + 8];
            if (c > 0) wait(L::PEmpty, c - 1);
#pragma unroll 1
            for (int J = 0; J <= w; ++J) {  // 16 columns; a loop that is not unrolled, see wait_longer
                float x[2][4];
                ptx::tmem_ld_frag2(lanes + kTmQk + (c & 1) * C + 16 * J, reinterpret_cast<uint32_t *>(x[0]));
                ptx::tmem_ld_wait();
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float *d = x[n];
                    const int col = 16 * J + 8 * n + 2 * tq;
                    const float4 Gc = *reinterpret_cast<const float4 *>(&g.G[col]);
                    const float2 a = make_float2(Gc.x, Gc.y), b = make_float2(Gc.z, Gc.w);
                    d[0] = r0 >= col ? d[0] * exp2_between(G0, a) : 0.f;
                    d[1] = r0 > col ? d[1] * exp2_between(G0, b) : 0.f;
                    d[2] = r0 + 8 >= col ? d[2] * exp2_between(G1, a) : 0.f;
                    d[3] = r0 + 8 > col ? d[3] * exp2_between(G1, b) : 0.f;
                    split(d[0], d[1], hi[2 * n], lo[2 * n]);
                    split(d[2], d[3], hi[2 * n + 1], lo[2 * n + 1]);
                }
                const uint32_t at = put_at + gdr::tile_off<128>(row, 16 * J + col8);
                store_matrices(at, hi);
                store_matrices(at + kHalf, lo);
            }
            ptx::tc_fence_before();
            warp_arrive(bar(L::QkEmpty + (c & 1)));
            ptx::fence_proxy_async();
            warp_arrive(bar(L::PFull));
            warp_arrive(bar(L::GEmpty + c % L::kGates));
            if (c + 1 < nc) keys(c + 1);
        }
    } else if (warp < 16) {
        constexpr int NC = DK / 2;  // key channels of a thread
        const int dv = (warp & 3) * 32 + lane, part = (warp - 8) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        float st[NC];
        const bool cut = sg.index > 0 || !sg.last;
        gdr::wait_for_previous_kernel();
        if (cut) {
            load_state<NC>(st, plan.states + ((size_t)slot * p.n_heads + head) * state_floats(DK), dv, part * NC);
        } else {
            load_given<NC>(st, p.h0 ? p.h0 + state_at : nullptr, p.d_k, p.d_v, dv, part * NC);
        }
        auto write_planes = [&] {
#pragma unroll
            for (int i = 0; i < NC; i += 16) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) split(st[i + 2 * j], st[i + 2 * j + 1], hi[j], lo[j]);
                ptx::tmem_st8(lanes + kTmS + (part * NC + i) / 2, hi);
                ptx::tmem_st8(lanes + kTmS + DK / 2 + (part * NC + i) / 2, lo);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            warp_arrive(bar(L::SFull));
        };
        write_planes();
        for (int c = 0; c < nc; ++c) {
            if (c + 1 == nc && !keep_end) break;
            wait(L::GFull + c % L::kGates, c / L::kGates);
            const float whole = gate(c)->whole;
            warp_arrive(bar(L::GEmpty + c % L::kGates));
            wait(L::DsFull, c);
            ptx::tc_fence_after();
#pragma unroll
            for (int i = 0; i < NC; i += 16) {
                float d[16];
                ptx::tmem_ld16(lanes + kTmDs + part * NC + i, reinterpret_cast<uint32_t *>(d));
                ptx::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) st[i + j] = fmaf(whole, st[i + j], d[j]);
            }
            ptx::tc_fence_before();
            warp_arrive(bar(L::DsEmpty));
            if (c + 1 == nc) break;
            wait(L::SEmpty, c);
            ptx::tc_fence_after();
            write_planes();
        }
        if (keep_end) store_given<NC>(st, p.h_final + state_at, p.d_k, p.d_v, dv, part * NC);
    } else {
        const int w = warp - 16, tq = lane & 3, ot = tid - 512;
        const bool live = 32 * w < p.d_v;
        const int64_t row_stride = (int64_t)p.n_heads * p.d_v;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + sg.t0 * row_stride + (int64_t)head * p.d_v;
        const int ch = (ot & 15) * 8;  // copied out: eight channels of every eighth token
        for (int c = 0; c < nc; ++c) {
            const TileGates &g = *gate(c);
            wait(L::GFull + c % L::kGates, c / L::kGates);
            // 16 value channels x 32 tokens a time; O1 leaves tensor memory first
            float o[4][4][4];
            wait(L::SEmpty, c);  // O1 is formed
            ptx::tc_fence_after();
            if (live) {
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    ptx::tmem_ld_frag4(tmem + ((uint32_t)(32 * w + 16 * (h & 1)) << 16) + kTmO1 + 32 * (h >> 1),
                                       reinterpret_cast<uint32_t *>(o[h][0]));
                ptx::tmem_ld_wait();
            }
            ptx::tc_fence_before();
            warp_arrive(bar(L::O1Empty));
            if (live)
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float2 gam = *reinterpret_cast<const float2 *>(&g.gam[32 * (h >> 1) + 8 * n + 2 * tq]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[h][n][e] *= e & 1 ? gam.y : gam.x;
                    }
            warp_arrive(bar(L::GEmpty + c % L::kGates));
            wait(L::O2Full, c);
            ptx::tc_fence_after();
            if (live)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int dv0 = 32 * w + 16 * (h & 1), tok0 = 32 * (h >> 1);
                    float b[4][4];
                    ptx::tmem_ld_frag4(tmem + ((uint32_t)dv0 << 16) + kTmO2 + tok0, reinterpret_cast<uint32_t *>(b[0]));
                    ptx::tmem_ld_wait();
                    uint32_t f[8];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) b[n][e] = p.scale * (o[h][n][e] + b[n][e]);
                        f[2 * n] = ptx::pack_bf16(b[n][0], b[n][1]);
                        f[2 * n + 1] = ptx::pack_bf16(b[n][2], b[n][3]);
                    }
#pragma unroll
                    for (int n = 0; n < 4; n += 2) {
                        const int tok = tok0 + 8 * n + (lane >> 4) * 8 + (lane & 7), at = dv0 + ((lane >> 3) & 1) * 8;
                        store_matrices_t(base + L::O + gdr::key_off(tok, at), f + 2 * n);
                    }
                }
            ptx::tc_fence_before();
            warp_arrive(bar(L::O2Empty));
            ptx::named_sync(2, 128);
            const int rows = rows_of(c);
            __nv_bfloat16 *to = out + ((int64_t)c * C + (ot >> 4)) * row_stride + ch;
            if (ch < p.d_v)
#pragma unroll
                for (int i = 0; i < 8; ++i, to += 8 * row_stride) {
                    const int r = (ot >> 4) + 8 * i;
                    if (r >= rows) break;
                    const uint4 x = *reinterpret_cast<const uint4 *>(smem + L::O + gdr::key_off(r, ch));
                    if (wide_out) {
                        *reinterpret_cast<uint4 *>(to) = x;
                    } else {
                        const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (ch + j < p.d_v) reinterpret_cast<uint16_t *>(to)[j] = (uint16_t)(e[j >> 1] >> (16 * (j & 1)));
                    }
                }
            ptx::named_sync(2, 128);
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 0) ptx::tmem_dealloc(tmem, 512);
}

template <int DK>
cudaError_t forward(const DlaArgs &p, cudaStream_t stream) {
    CUtensorMap q, k, v;
    const bool copies = TileMap::encode(&q, p.q, p.n_tok, p.q_stride, p.n_k_heads, p.d_k) &&
                        TileMap::encode(&k, p.k, p.n_tok, p.k_stride, p.n_k_heads, p.d_k) &&
                        TileMap::encode(&v, p.v, p.n_tok, p.v_stride, p.n_heads, p.d_v);
    const bool wide = p.d_v % 8 == 0 && (uintptr_t)p.out % 16 == 0;
    Plan plan = make_plan(p, false);
    const unsigned blocks = (unsigned)(plan.slots * p.n_heads);
    if (plan.cut) {
        const cudaError_t e = launch_segments<DK>(p, plan, q, k, v, v, copies, false, stream);
        if (e != cudaSuccess) return e;
        return gdr::launch_dependent(dla_forward_kernel<DK>, dim3(blocks), kFwdThreads, FwdSmem<DK>::kBytes, stream, q, k, v, p,
                                     plan, copies, wide);
    }
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(dla_forward_kernel<DK>), FwdSmem<DK>::kBytes);
    if (e != cudaSuccess) return e;
    dla_forward_kernel<DK><<<blocks, kFwdThreads, FwdSmem<DK>::kBytes, stream>>>(q, k, v, p, plan, copies, wide);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace
}  // namespace dla

size_t dla_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t, int32_t d_k, int32_t d_v, bool bf16,
                           bool bwd) {
    if (bf16 && !bwd) return dla_tc_fwd_workspace_bytes(n_tok, n_seq, n_heads, d_k);
    return dla_simt_workspace_bytes(n_tok, n_seq, n_heads, d_k, d_v, bwd);
}
cudaError_t launch_dla_fwd(const DlaArgs &p, cudaStream_t stream) {
    return p.bf16 && p.n_tok > 0 ? launch_dla_tc_fwd(p, stream) : launch_dla_simt(p, false, stream);
}
cudaError_t launch_dla_bwd(const DlaArgs &p, cudaStream_t stream) { return launch_dla_simt(p, true, stream); }

size_t dla_tc_fwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t d_k) {
    return dla::plan_bytes(n_tok, n_seq, n_heads, d_k, false);
}

cudaError_t launch_dla_tc_fwd(const DlaArgs &p, cudaStream_t stream) {
    return p.d_k <= 64 ? dla::forward<64>(p, stream) : dla::forward<128>(p, stream);
}

cudaError_t read_dla_fwd_flags(unsigned int *flags, bool reset, cudaStream_t stream) {
    return dla::read_flags(flags, reset, stream);
}

}  // namespace kda
