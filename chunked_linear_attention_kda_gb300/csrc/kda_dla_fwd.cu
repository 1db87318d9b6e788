// kda_dla_fwd.cu -- chunked forward of linear attention with one decay per head, bf16 inputs, on
// tcgen05; the formulas are in kda_dla.h.
//
// A CTA walks over a segment of one sequence and head in tiles of 64 tokens and carries the state
// S^T (d_v x d_k, fp32, in the registers of eight warps). Per tile, with tokens as columns so that
// every product has 128 rows:
//   Q K^T                        64 x 64, both tiles as they were copied
//   O1 = S^T Q^T                 S^T as two bf16 planes in tensor memory (the A operand)
//   O2 = V^T P^T                 P = scale e Q K^T as two planes in shared memory
//   dS^T = V'^T K                V' = delta V as two planes in tensor memory: a tile's sums are off by 4e-6
//                                of their norm, a thousandth of what a bf16 input is rounded by; with a third
//                                plane Q K^T has room for one tile, and this launch takes 517 us instead
//                                of 400 at 64K tokens of 32 heads
//   o = scale gamma O1 + O2,  S^T <- Gamma S^T + dS^T
// The state is converted once a tile, off the products' path: what waits for it is O1 alone. Shared
// memory's 128 bytes a cycle bound a tile (the operands of the products, V' and P formed, the output
// turned): what can be is an A operand in tensor memory.
//
// A long sequence is cut into segments, so that few heads fill the GPU: a first launch forms what
// each segment adds to the state (kda_dla_states.h: K and V are read once more), a second one the
// states at the segments' starts, a third the output, all segments side by side. 64K tokens of 32 heads, 128 x
// 128, 630 us: under the profiler gates 17 us, segments 172 us (1.07 GB, 0.93 of the copy rate), join 12 us, output
// 390 us (2.15 GB, 0.83 of it; 3500 cycles a tile, with no unit above half: the roles of a tile wait for one another).
#include <cmath>

#include "kda_dla_states.h"

namespace kda {
namespace dla {
namespace {

// warps: 0 and 1 issue products, 2 and 3 load, 4..7 scale values, 8..15 form P, 16..23 hold the state, 24..31 the output
constexpr int kFwdThreads = 1024;
// Registers a thread has at launch, and each warpgroup's after it gave away or took some: together what
// the block was launched with.
constexpr int kRegsLaunch = 64, kRegsServe = 40, kRegsPairs = 56, kRegsState = 96, kRegsOut = 64;
static_assert(2 * (kRegsServe + kRegsPairs + kRegsState + kRegsOut) == 8 * kRegsLaunch, "the launch's registers");

// Queries and keys of a tile are free once their products are done, its values when the output that was
// turned in their place is copied out, its gates after all of it: rings of their own. A tile takes 4000
// cycles to arrive, and with one ring of three stages that was waited for.
template <int DK>
struct FwdSmem {
    static constexpr int kKey = DK / 64 * kHalf, kVal = 2 * kHalf;
    static constexpr int kStages = 4, kGates = 6;
    static constexpr int Q = 0, K = kKey, kPair = 2 * kKey;  // a stage of queries and keys
    static constexpr int V = kStages * kPair, P = V + kStages * kVal, Gate = P + 2 * kHalf, Bars = Gate + kGates * (int)sizeof(TileGates);
    // rings' full and empty, then one each, but those of QK and O2, which alternate: either may be formed a
    // tile before the last one was seen, and a phase's parity tells neighbours apart only
    static constexpr int KFull = 0, KEmpty = KFull + kStages, VFull = KEmpty + kStages, VEmpty = VFull + kStages,
                         GFull = VEmpty + kStages, GEmpty = GFull + kGates, QkFull = GEmpty + kGates, PFull = QkFull + 2,
                         PEmpty = PFull + 1, VpFull = PEmpty + 1, VpEmpty = VpFull + 1, DsFull = VpEmpty + 1,
                         DsEmpty = DsFull + 1, SFull = DsEmpty + 1, O1Full = SFull + 1, O1Empty = O1Full + 1,
                         O2Full = O1Empty + 1, O2Empty = O2Full + 2, Drain = O2Empty + 2, Partial = Drain + 2, kBars = Partial + 2;
    static constexpr int kBytes = Bars + 8 * kBars + 16 + 1024;  // the base is rounded up to 1024
    static_assert(kBytes <= 227 * 1024, "fits an SM");
};
// columns of tensor memory
constexpr int kTmDs = 0, kTmS = 128, kTmO1 = 256, kTmV = 320, kTmQk = 384;  // kTmQk: Q K^T, then O2, of two tiles

// OWN: the gates are formed here, by a loading warp (short calls; apart, because the rest takes 1.3 times as
// long with that code beside it)
template <int DK, bool OWN>
__global__ void __launch_bounds__(kFwdThreads, 1)
    dla_forward_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const DlaArgs p, const Plan plan, bool copies,
                       bool wide_out) {
    using L = FwdSmem<DK>;
    constexpr int S = L::kStages;
    extern __shared__ __align__(1024) char smem_raw[];
    char *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    // equal over a warp, and told to the compiler so: branches and loops on them keep operands in
    // uniform registers
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int head = blockIdx.x % p.n_heads, kh = head / (p.n_heads / p.n_k_heads);
    const Ordered unit = jth_longest(p.cu_seqlens, p.n_seq, blockIdx.x / p.n_heads, plan.slots, plan.seg, smem);
    const int64_t slot = unit.slot;
    const Segment sg = unit.sg;
    const int64_t state_at = ((int64_t)sg.seq * p.n_heads + head) * p.d_k * p.d_v;
    if (sg.len == 0) {
        gdr::wait_for_previous_kernel();  // whoever waits for this kernel waits for that one
        if (sg.last && p.h_final)  // an empty sequence
            for (int i = tid; i < p.d_k * p.d_v; i += kFwdThreads) p.h_final[state_at + i] = p.h0 ? p.h0[state_at + i] : 0.f;
        return;
    }
    const int nc = uniform((int)((sg.len + C - 1) / C));
    const bool keep_end = uniform(sg.last) && p.h_final;  // else the last tile adds to no state
    auto bar = [&](int i) { return base + L::Bars + 8 * i; };
    auto gate = [&](int c) -> const TileGates & {
        return reinterpret_cast<const TileGates *>(smem + L::Gate)[c % L::kGates];
    };
    auto rows_of = [&](int c) { return (int)min((int64_t)C, sg.len - (int64_t)c * C); };

    // the state's lines are asked for while the block sets itself up
    if (p.h0 && sg.index == 0 && sg.last && tid * 32 < p.d_k * p.d_v)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.h0 + state_at + tid * 32));
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            ptx::mbar_init(bar(L::KFull + i), 1);
            ptx::mbar_init(bar(L::KEmpty + i), 2);
            ptx::mbar_init(bar(L::VFull + i), 1);
            ptx::mbar_init(bar(L::VEmpty + i), 8);
        }
        for (int i = 0; i < L::kGates; ++i) {
            ptx::mbar_init(bar(L::GFull + i), 1);
            ptx::mbar_init(bar(L::GEmpty + i), 4 + 8 + 8 + 8);  // values, P, state, output
        }
        ptx::mbar_init(bar(L::QkFull), 1);
        ptx::mbar_init(bar(L::QkFull + 1), 1);
        ptx::mbar_init(bar(L::PFull), 8);
        ptx::mbar_init(bar(L::PEmpty), 1);
        ptx::mbar_init(bar(L::VpFull), 4);
        ptx::mbar_init(bar(L::VpEmpty), 1);
        ptx::mbar_init(bar(L::DsFull), 1);
        ptx::mbar_init(bar(L::DsEmpty), 8);
        ptx::mbar_init(bar(L::SFull), 8);
        ptx::mbar_init(bar(L::O1Full), 1);
        ptx::mbar_init(bar(L::O1Empty), 8);
        ptx::mbar_init(bar(L::O2Full), 1);
        ptx::mbar_init(bar(L::O2Full + 1), 1);
        ptx::mbar_init(bar(L::O2Empty), 8);
        ptx::mbar_init(bar(L::O2Empty + 1), 8);
        ptx::mbar_init(bar(L::Drain), 1);
        ptx::mbar_init(bar(L::Drain + 1), 1);
        ptx::mbar_init(bar(L::Partial), 1);
        ptx::mbar_init(bar(L::Partial + 1), 1);
        ptx::mbar_init_fence();
    }
    if (warp == 0) ptx::tmem_alloc(bar(L::kBars), 512);
    // P is zero above its diagonal blocks
    for (int i = tid; i < 2 * kHalf / 16; i += kFwdThreads) reinterpret_cast<uint4 *>(smem + L::P)[i] = make_uint4(0, 0, 0, 0);
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
        ptx::regs_decrease<kRegsServe>();
        // Q K^T a tile ahead, and O1 (in the other order the next tile's P waits for this one's state: 445 -> 463 us
        // at 64K tokens of 32 heads). Two warps issue, because a product takes its warp 40 to 70 cycles to issue
        // and a tile has 40 of them. The whole warp walks, an elected lane issues: operands are formed in
        // uniform registers.
        constexpr uint32_t id_qk = ptx::idesc_bf16(64, C, 0, 0), id_o1 = ptx::idesc_bf16(128, C, 0, 0);
        const uint32_t leader = ptx::elect_one();
        const uint64_t q0 = ptx::sdesc_sw128(base + L::Q, 16, 1024), k0 = ptx::sdesc_sw128(base + L::K, 16, 1024);
        auto step = [](int k) { return (uint32_t)((k >> 2) * kHalf + (k & 3) * 32) / 16; };  // 16 channels, K-major
        int next = 0, next_phase = 0;  // the stage of the next Q K^T
        int s = 0;
#pragma unroll 1
        for (int c = -1; c < nc; ++c) {
            if (c + 1 < nc) {
                wait(L::KFull + next, next_phase);
                if (c >= 1) wait(L::O2Empty + ((c + 1) & 1), (c - 1) >> 1);  // the columns
                ptx::tc_fence_after();
                const uint32_t at = (uint32_t)next * (L::kPair / 16);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)
                        ptx::umma_ss(tmem + kTmQk + ((c + 1) & 1) * C, q0 + (at + step(k)), k0 + (at + step(k)), id_qk, k > 0);
                    ptx::umma_commit(bar(L::QkFull + ((c + 1) & 1)));
                }
                __syncwarp();
                if (++next == S) {
                    next = 0;
                    next_phase ^= 1;
                }
            }
            if (c >= 0) {
                wait(L::SFull, c);
                if (c > 0) wait(L::O1Empty, c - 1);
                ptx::tc_fence_after();
                const uint32_t at = (uint32_t)s * (L::kPair / 16);
                if (leader) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < DK / 16; ++k)
                            ptx::umma_ts(tmem + kTmO1, tmem + kTmS + i * (DK / 2) + 8 * k, q0 + (at + step(k)), id_o1, i + k > 0);
                    ptx::umma_commit(bar(L::O1Full));
                    ptx::umma_commit(bar(L::KEmpty + s));
                }
                __syncwarp();
                if (++s == S) s = 0;
            }
        }
        if (leader) ptx::umma_commit(bar(L::Drain));
        __syncwarp();
        drain_bar(bar(L::Drain), 0);
    } else if (warp == 1) {
        ptx::regs_decrease<kRegsServe>();
        // dS^T and O2
        constexpr uint32_t id_o2 = ptx::idesc_bf16(128, C, 1, 0), id_ds = ptx::idesc_bf16(128, DK, 0, 1);
        const uint32_t leader = ptx::elect_one();
        const uint64_t v0 = ptx::sdesc_sw128(base + L::V, kHalf, 1024), k0 = ptx::sdesc_sw128(base + L::K, kHalf, 1024);
        const uint64_t pp = ptx::sdesc_sw128(base + L::P, 16, 1024);
        int s = 0;
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
            const uint32_t at = (uint32_t)s * (L::kVal / 16), key = (uint32_t)s * (L::kPair / 16);
            wait(L::KFull + s, c / S);
            wait(L::VFull + s, c / S);
            if (c + 1 < nc || keep_end) {
                wait(L::VpFull, c);
                if (c > 0) wait(L::DsEmpty, c - 1);
                ptx::tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int i = 1; i >= 0; --i)
#pragma unroll
                        for (int k = 0; k < C / 16; ++k)
                            ptx::umma_ts(tmem + kTmDs, tmem + kTmV + i * 32 + 8 * k, k0 + (key + 128 * k), id_ds, i < 1 || k > 0);
                    ptx::umma_commit(bar(L::DsFull));
                    ptx::umma_commit(bar(L::VpEmpty));
                    ptx::umma_commit(bar(L::KEmpty + s));
                }
                __syncwarp();
            }
            wait(L::PFull, c);
            ptx::tc_fence_after();
            if (leader) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int k = 0; k < C / 16; ++k)
                        ptx::umma_ss(tmem + kTmQk + (c & 1) * C, v0 + (at + 128 * k), pp + (i * kHalf + k * 32) / 16, id_o2, i + k > 0);
                ptx::umma_commit(bar(L::O2Full + (c & 1)));
                ptx::umma_commit(bar(L::PEmpty));
            }
            __syncwarp();
            if (++s == S) s = 0;
        }
        if (leader) ptx::umma_commit(bar(L::Drain + 1));
        __syncwarp();
        drain_bar(bar(L::Drain + 1), 0);
    } else if (warp < 4) {
        ptx::regs_decrease<kRegsServe>();
        // one loads keys, queries and gates, the other values
        const bool pair = warp == 2;
        const Source in[2] = {
            {pair ? &tm_k : &tm_v, static_cast<const __nv_bfloat16 *>(pair ? p.k : p.v), pair ? p.k_stride : p.v_stride, pair ? kh : head,
             pair ? p.in_k : p.in_v, pair ? DK / 64 : p.d_v > 64 ? 2 : 1, pair ? plan.vec_k : plan.vec_v},
            {&tm_q, static_cast<const __nv_bfloat16 *>(p.q), p.q_stride, kh, p.in_k, DK / 64, plan.vec_q}};
        const TileGates *gates = gates_of(plan.gates, p, sg.seq, (int64_t)sg.index * (plan.seg / C), head);
        const int full = pair ? L::KFull : L::VFull, empty = pair ? L::KEmpty : L::VEmpty;
        int begun = 0;  // tiles whose copies were begun
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
            const int s = c % S, rows = rows_of(c);
            if (c >= S) wait(empty + s, c / S - 1);
            if (pair && c >= L::kGates) wait(L::GEmpty + c % L::kGates, c / L::kGates - 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t to[2] = {base + (pair ? s * L::kPair + L::K : L::V + s * L::kVal), base + s * L::kPair + L::Q};
            const int64_t t0 = sg.t0 + (int64_t)c * C;
            const uint32_t m = bar(full + s);
            if (copies) {
                // a partial tile is copied whole; what is another sequence's goes before it is handed over
                const uint32_t by = rows == C ? m : bar(L::Partial + (pair ? 0 : 1));
                if (lane == 0) {
                    ptx::mbar_arrive_tx(by, pair ? 2 * L::kKey : in[0].halves * kHalf);
                    tile_by_copy(in[0], to[0], t0, by);
                    if (pair) tile_by_copy(in[1], to[1], t0, by);
                }
                if (rows < C) {  // the walk's last
                    if (!wait_bar(by, 0)) drain_bar(by, 0);
                    clear_rows(to[0], in[0].halves, kHalf, rows, C);
                    if (pair) clear_rows(to[1], in[1].halves, kHalf, rows, C);
                    ptx::fence_proxy_async();
                    warp_arrive(m);
                }
            } else {
                tiles_by_threads(in, to, pair ? 2 : 1, t0, rows, lane, 32);
                rows_loaded();
                if (lane == 0) ptx::mbar_arrive(m);
            }
            if (OWN && pair) {
                const int r = 2 * lane;
                const float *g = p.g + (t0 + r) * p.g_stride + head;
                form_gates(make_float2(r < rows ? g[0] : 0.f, r + 1 < rows ? g[p.g_stride] : 0.f), p.scale,
                           reinterpret_cast<TileGates *>(smem + L::Gate) + c % L::kGates);
                warp_arrive(bar(L::GFull + c % L::kGates));
            } else if (pair && lane == 0) {
                if (c == 0) gdr::wait_for_previous_kernel();  // the gates
                const uint32_t gm = bar(L::GFull + c % L::kGates);
                ptx::mbar_arrive_tx(gm, sizeof(TileGates));
                bulk_load(base + L::Gate + c % L::kGates * (uint32_t)sizeof(TileGates), gates + (int64_t)c * p.n_heads, sizeof(TileGates), gm);
            }
            begun = c + 1;
        }
        // nothing may land in shared memory after the block has gone
        if (!ok) {
            for (int c = max(0, begun - S); c < begun; ++c) drain_bar(bar(full + c % S), (c / S) & 1);
            if (pair && !OWN)
                for (int c = max(0, begun - L::kGates); c < begun; ++c) drain_bar(bar(L::GFull + c % L::kGates), (c / L::kGates) & 1);
        }
    } else if (warp < 8) {
        ptx::regs_decrease<kRegsServe>();
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
            if (c + 1 == nc && !keep_end) break;  // adds to no state
            const int s = c % S;
            wait(L::GFull + c % L::kGates, c / L::kGates);
            wait(L::VFull + s, c / S);
            auto ready = [&] {
                if (c > 0) wait(L::VpEmpty, c - 1);
                ptx::tc_fence_after();
            };
            if (32 * (warp & 3) < p.d_v) scale_values<2>(base + L::V + s * L::kVal, tmem, kTmV, gate(c).del, 1.f, ready);
            else ready();
            ptx::tc_fence_before();
            warp_arrive(bar(L::VpFull));
            warp_arrive(bar(L::GEmpty + c % L::kGates));
        }
    } else if (warp < 16) {
        ptx::regs_decrease<kRegsPairs>();
        // 16 rows by two warps, which take turns at its blocks of 16 columns
        const int w = warp & 3, J0 = (warp - 8) >> 2, gr = lane >> 2, tq = lane & 3;
        const uint32_t lanes = tmem + ((uint32_t)(w * 32) << 16);
        const uint32_t put_at = base + L::P, row = 16 * w + ((lane >> 3) & 1) * 8 + (lane & 7), col8 = (lane >> 4) * 8;
        const int r0 = 16 * w + gr;
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
            wait(L::GFull + c % L::kGates, c / L::kGates);
            const TileGates &g = gate(c);
            const float2 G0 = g.G[r0], G1 = g.G[r0 + 8];
            wait(L::QkFull + (c & 1), c >> 1);
            if (c > 0) wait(L::PEmpty, c - 1);
            ptx::tc_fence_after();
#pragma unroll 1
            for (int J = J0; J <= w; J += 2) {  // a loop that is not unrolled: warps wait for instructions
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
                    d[0] = r0 >= col ? p.scale * d[0] * exp2_between(G0, a) : 0.f;
                    d[1] = r0 > col ? p.scale * d[1] * exp2_between(G0, b) : 0.f;
                    d[2] = r0 + 8 >= col ? p.scale * d[2] * exp2_between(G1, a) : 0.f;
                    d[3] = r0 + 8 > col ? p.scale * d[3] * exp2_between(G1, b) : 0.f;
                    split(d[0], d[1], hi[2 * n], lo[2 * n]);
                    split(d[2], d[3], hi[2 * n + 1], lo[2 * n + 1]);
                }
                const uint32_t at = put_at + gdr::tile_off<128>(row, 16 * J + col8);
                store_matrices(at, hi);
                store_matrices(at + kHalf, lo);
            }
            ptx::tc_fence_before();
            ptx::fence_proxy_async();
            warp_arrive(bar(L::PFull));
            warp_arrive(bar(L::GEmpty + c % L::kGates));
        }
    } else if (warp < 24) {
        ptx::regs_increase<kRegsState>();
        constexpr int NC = DK / 2;  // key channels of a thread
        const int dv = (warp & 3) * 32 + lane, part = (warp - 16) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        // Lanes of channels that no value has hold what they will: a product's row depends on its own lane
        // alone, and theirs are not read.
        const bool live = 32 * (warp & 3) < p.d_v;
        float st[NC];
        const bool cut = sg.index > 0 || !sg.last;
        Factors decays;
        gdr::wait_for_previous_kernel();
        if (cut) load_state<NC>(st, plan.states + ((size_t)slot * p.n_heads + head) * state_floats(DK), dv, part * NC);
        else load_given<NC>(st, p.h0 ? p.h0 + state_at : nullptr, p.d_k, p.d_v, dv, part * NC);
#pragma unroll 1
        for (int c = 0;; ++c) {
            if (c > 0) {
                wait(L::O1Full, c - 1);  // the last planes are read
                ptx::tc_fence_after();
            }
            if (live)
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
            if (c + 1 == nc && !keep_end) break;
            wait(L::GFull + c % L::kGates, c / L::kGates);
            const float whole = decays.next(gate(c).whole);
            warp_arrive(bar(L::GEmpty + c % L::kGates));
            wait(L::DsFull, c);
            ptx::tc_fence_after();
            if (live)
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
        }
        if (keep_end) store_given<NC>(st, p.h_final + state_at, p.d_k, p.d_v, dv, part * NC);
    } else {
        // 32 value channels x 32 tokens a warp
        const int w = warp & 3, tok0 = 32 * ((warp - 24) >> 2), tq = lane & 3, ot = tid - 768;
        const bool live = 32 * w < p.d_v;
        const int64_t row_stride = (int64_t)p.n_heads * p.d_v;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + sg.t0 * row_stride + (int64_t)head * p.d_v;
        const int ch = (ot & 15) * 8;  // copied out: eight channels of every sixteenth token
        const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16) + tok0;
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
            const uint32_t stage = L::V + c % S * L::kVal;  // in the place of the tile's values
            wait(L::GFull + c % L::kGates, c / L::kGates);
            const TileGates &g = gate(c);
            // O1 leaves tensor memory first
            float o[2][4][4];
            wait(L::O1Full, c);
            ptx::tc_fence_after();
            if (live) {
                ptx::tmem_ld_frag4(lanes + kTmO1, reinterpret_cast<uint32_t *>(o[0][0]));
                ptx::tmem_ld_frag4(lanes + (16u << 16) + kTmO1, reinterpret_cast<uint32_t *>(o[1][0]));
                ptx::tmem_ld_wait();
            }
            ptx::tc_fence_before();
            warp_arrive(bar(L::O1Empty));
            wait(L::O2Full + (c & 1), c >> 1);
            ptx::tc_fence_after();
            if (live)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float b[4][4];
                    ptx::tmem_ld_frag4(lanes + ((uint32_t)(16 * h) << 16) + kTmQk + (c & 1) * C, reinterpret_cast<uint32_t *>(b[0]));
                    ptx::tmem_ld_wait();
                    uint32_t f[8];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float2 gam = *reinterpret_cast<const float2 *>(&g.gam[tok0 + 8 * n + 2 * tq]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) b[n][e] = fmaf(e & 1 ? gam.y : gam.x, o[h][n][e], b[n][e]);
                        f[2 * n] = ptx::pack_bf16(b[n][0], b[n][1]);
                        f[2 * n + 1] = ptx::pack_bf16(b[n][2], b[n][3]);
                    }
#pragma unroll
                    for (int n = 0; n < 4; n += 2) {
                        const int tok = tok0 + 8 * n + (lane >> 4) * 8 + (lane & 7), at = 32 * w + 16 * h + ((lane >> 3) & 1) * 8;
                        store_matrices_t(base + stage + gdr::key_off(tok, at), f + 2 * n);
                    }
                }
            ptx::tc_fence_before();
            warp_arrive(bar(L::O2Empty + (c & 1)));
            warp_arrive(bar(L::GEmpty + c % L::kGates));
            ptx::named_sync(2, 256);
            const int rows = rows_of(c);
            __nv_bfloat16 *to = out + ((int64_t)c * C + (ot >> 4)) * row_stride + ch;
            if (ch < p.d_v)
#pragma unroll
                for (int i = 0; i < 4; ++i, to += 16 * row_stride) {
                    const int r = (ot >> 4) + 16 * i;
                    if (r >= rows) break;
                    const uint4 x = *reinterpret_cast<const uint4 *>(smem + stage + gdr::key_off(r, ch));
                    if (wide_out) {
                        *reinterpret_cast<uint4 *>(to) = x;
                    } else {
                        const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (ch + j < p.d_v) reinterpret_cast<uint16_t *>(to)[j] = (uint16_t)(e[j >> 1] >> (16 * (j & 1)));
                    }
                }
            ptx::fence_proxy_async();  // the next tile is copied there
            warp_arrive(bar(L::VEmpty + c % S));
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 0) ptx::tmem_dealloc(tmem, 512);
}

template <int DK>
cudaError_t forward(const DlaArgs &p, cudaStream_t stream) {
    CUtensorMap q, k, v;
    const bool copies = TileMap::encode(&q, p.q, p.n_tok, p.q_stride, p.n_k_heads, p.in_k) &&
                        TileMap::encode(&k, p.k, p.n_tok, p.k_stride, p.n_k_heads, p.in_k) &&
                        TileMap::encode(&v, p.v, p.n_tok, p.v_stride, p.n_heads, p.in_v);
    const bool wide = p.d_v % 8 == 0 && (uintptr_t)p.out % 16 == 0;
    const Plan plan = make_plan(p, false);
    // A short call forms the gates beside the tiles' copies: a launch less (40 tokens of 32 heads in a graph:
    // 8.7 us, 9.6 with the launch), but 2 us a tile that nothing hides.
    const dim3 grid((unsigned)(plan.slots * p.n_heads));
    if (p.n_tok <= 4 * C && !plan.cut) {
        const cudaError_t e = allow_smem(reinterpret_cast<const void *>(dla_forward_kernel<DK, true>), FwdSmem<DK>::kBytes);
        if (e != cudaSuccess) return e;
        dla_forward_kernel<DK, true><<<grid, kFwdThreads, FwdSmem<DK>::kBytes, stream>>>(q, k, v, p, plan, copies, wide);
        count_launches(1);
        return cudaGetLastError();
    }
    cudaError_t e = launch_gates(p, plan, stream);
    if (e == cudaSuccess && plan.cut) e = launch_segments<DK>(p, plan, q, k, v, v, copies, 1, stream);
    if (e != cudaSuccess) return e;
    return gdr::launch_dependent(dla_forward_kernel<DK, false>, grid, kFwdThreads, FwdSmem<DK>::kBytes, stream, q, k, v, p, plan, copies,
                                 wide);
}

}  // namespace
}  // namespace dla

size_t dla_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k, int32_t d_v,
                           bool bf16, bool bwd) {
    if (!bf16) return dla_simt_workspace_bytes(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v, bwd);
    return bwd ? dla_tc_bwd_workspace_bytes(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v)
               : dla_tc_fwd_workspace_bytes(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v);
}
// without a token the states pass through: nothing of bf16 is read
cudaError_t launch_dla_fwd(const DlaArgs &p, cudaStream_t stream) {
    return p.bf16 && p.n_tok > 0 ? launch_dla_tc_fwd(p, stream) : launch_dla_simt(p, false, stream);
}
cudaError_t launch_dla_bwd(const DlaArgs &p, cudaStream_t stream) {
    return p.bf16 && p.n_tok > 0 ? launch_dla_tc_bwd(p, stream) : launch_dla_simt(p, true, stream);
}

size_t dla_tc_fwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k, int32_t d_v) {
    return dla::plan_bytes(n_tok, n_seq, n_heads, d_k) + dla::copies_bytes(n_tok, n_heads, n_k_heads, d_k, d_v, false);
}

cudaError_t launch_dla_tc_fwd(const DlaArgs &args, cudaStream_t stream) {
    DlaArgs p = args;
    const cudaError_t e = dla::align_inputs(p, static_cast<char *>(p.workspace) + dla::plan_bytes(p.n_tok, p.n_seq, p.n_heads, p.d_k), false, stream);
    if (e != cudaSuccess) return e;
    return p.d_k <= 64 ? dla::forward<64>(p, stream) : dla::forward<128>(p, stream);
}

cudaError_t read_dla_fwd_flags(unsigned int *flags, bool reset, cudaStream_t stream) {
    return dla::read_flags(flags, reset, stream);
}

}  // namespace kda
