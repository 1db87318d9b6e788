// kda_dla_bwd.cu -- backward pass of chunked linear attention with one decay per head, bf16 inputs, on
// tcgen05; the formulas are in kda_dla.h, with a chunk of 128 tokens.
//
// Launches: the gates of every tile; (long sequences of few heads: what each segment adds to the state
// and to its gradient, and the join, as in the forward pass); a walk over every sequence's or
// segment's tiles in both directions that leaves the state at each block of 128 tokens' start and the
// gradient at its end in the workspace, as two bf16 planes that tensor copies of a block's gradients read;
// the gradients, every block and value head by itself; with shared heads the sums over value heads.
// Two sequences of 8K tokens, 32 heads, 128 x 128: gates 8 us, states 174 us (1.07 GB, 0.92 of the copy rate),
// gradients 338 us (1.45 GB, 0.64; a block is a chain of five products, 12 us). Blocks of 128 tokens, because
// their four products fill tensor memory and their tiles shared memory; blocks of 64 would keep twice
// the states, 1.07 GB more traffic.
#include <cmath>

#include "kda_dla_states.h"

namespace kda {
namespace dla {
namespace {

constexpr int kBlock = 128;  // tokens
constexpr int kWide = kBlock * 128;  // bytes of a tile's 64 channels

// ---------------------------------------------------------------- states
// Block b of sequence n lies in slot cu[n] / 128 + n + b.
__host__ __device__ __forceinline__ int64_t block_slots(int64_t n_tok, int64_t n_seq) { return n_tok / kBlock + n_seq; }
__device__ __forceinline__ int64_t block_base(const int32_t *cu, int n) { return (int64_t)(cu[n] >> 7) + n; }
// Per (slot, value head): the planes of S0^T, then those of dS1^T; a plane is DK / 64 parts of DV rows of
// 64 key channels in the 128-byte swizzle.
constexpr int plane_bytes(int dkp, int dvp) { return dkp * dvp * 2; }
__host__ __device__ __forceinline__ constexpr size_t pair_bytes(int dkp, int dvp) { return (size_t)4 * plane_bytes(dkp, dvp); }

struct BwdPlan {
    Plan walk;
    char *states;        // [block slots][heads] pair_bytes
    float *sums;         // [block slots][heads] sums of dg (one decay per head)
    float *dq, *dk;      // [tokens][heads][DK] parts of dq and dk (shared heads)
};

// warps: 0 issues products, 1 loads, 2 stores, 4..7 scale the values, 8..15 hold the state
constexpr int kWalkThreads = 512;

template <int DK, int DV>
struct WalkSmem {
    static constexpr int kKey = DK / 64 * kHalf, kVal = 2 * kHalf;
    static constexpr int K = 0, V = kKey, Gate = V + kVal, kStage = Gate + 2048;
    static constexpr int kStages = 4;
    static constexpr int Out = kStages * kStage, Bars = Out + 2 * plane_bytes(DK, DV);
    static constexpr int Full = 0, Empty = kStages, VpFull = 2 * kStages, VpEmpty = VpFull + 2, DsFull = VpEmpty + 2,
                         DsEmpty = DsFull + 2, OutFull = DsEmpty + 2, OutEmpty = OutFull + 1, Drain = OutEmpty + 1, Partial = Drain + 1, kBars = Partial + 1;
    static constexpr int kBytes = Bars + 8 * kBars + 16 + 1024;  // the base is rounded up to 1024
    static_assert(sizeof(TileGates) <= 2048 && kBytes <= 227 * 1024, "fits an SM");
};

template <int DK, int DV, bool REV>
__device__ __forceinline__ void state_walk(const CUtensorMap &tm_key, const CUtensorMap &tm_val, const DlaArgs &p,
                                           const BwdPlan &bp, bool copies, unsigned unit) {
    using L = WalkSmem<DK, DV>;
    constexpr int S = L::kStages;
    extern __shared__ __align__(1024) char smem_raw[];
    char *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    const Plan &plan = bp.walk;
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };  // equal over a warp, and told so
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int head = unit % p.n_heads, kh = head / (p.n_heads / p.n_k_heads);
    const Ordered mine = jth_longest(p.cu_seqlens, p.n_seq, unit / p.n_heads, plan.slots, plan.seg, smem);
    const int64_t slot = mine.slot;
    const Segment sg = mine.sg;
    const int64_t state_at = ((int64_t)sg.seq * p.n_heads + head) * p.d_k * p.d_v;
    if (sg.len == 0) {
        if (REV && sg.last && p.dh0)  // an empty sequence
            for (int i = tid; i < p.d_k * p.d_v; i += kWalkThreads) p.dh0[state_at + i] = p.dh_final ? p.dh_final[state_at + i] : 0.f;
        gdr::wait_for_previous_kernel();  // whoever waits for this kernel waits for that one
        return;
    }
    const int nc = uniform((int)((sg.len + C - 1) / C));
    // the walk's last step is left out where nothing reads its sum
    const int steps = REV ? (sg.index == 0 && p.dh0 ? nc : nc - 1) : nc - 1;
    auto bar = [&](int i) { return base + L::Bars + 8 * i; };
    auto tile = [&](int n) { return REV ? nc - 1 - n : n; };  // the n-th of the walk
    auto rows_of = [&](int c) { return (int)min((int64_t)C, sg.len - (int64_t)c * C); };
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            ptx::mbar_init(bar(L::Full + i), 1);
            ptx::mbar_init(bar(L::Empty + i), 1 + 4 + 8);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(L::VpFull + i), 4);
            ptx::mbar_init(bar(L::VpEmpty + i), 1);
            ptx::mbar_init(bar(L::DsFull + i), 1);
            ptx::mbar_init(bar(L::DsEmpty + i), 8);
        }
        ptx::mbar_init(bar(L::OutFull), 8);
        ptx::mbar_init(bar(L::OutEmpty), 1);
        ptx::mbar_init(bar(L::Drain), 1);
        ptx::mbar_init(bar(L::Partial), 1);
        ptx::mbar_init_fence();
    }
    if (warp == 0) ptx::tmem_alloc(bar(L::kBars), 512);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<const uint32_t *>(smem + L::Bars + 8 * L::kBars);
    bool ok = true;
    auto wait = [&](int b, int parity) { ok = wait_bar(bar(b), parity & 1) && ok; };
    // a block's state is kept before the walk enters it
    auto enters = [&](int n) { return REV ? (tile(n) & 1) || n == 0 : (tile(n) & 1) == 0; };
    if (warp == 0) {
        constexpr uint32_t id = ptx::idesc_bf16(128, DK, 0, 1);
        const uint32_t leader = ptx::elect_one();
        const uint64_t k0 = ptx::sdesc_sw128(base + L::K, kHalf, 1024);
        int s = 0;
#pragma unroll 1
        for (int n = 0; n < steps; ++n) {
            wait(L::VpFull + (n & 1), n >> 1);
            if (n >= 2) wait(L::DsEmpty + (n & 1), (n >> 1) - 1);
            ptx::tc_fence_after();
            const uint32_t at = (uint32_t)s * (L::kStage / 16);
            if (leader) {
#pragma unroll
                for (int i = 2; i >= 0; --i)  // the smallest first
#pragma unroll
                    for (int k = 0; k < C / 16; ++k)
                        ptx::umma_ts(tmem + (n & 1) * 128, tmem + 256 + (n & 1) * 96 + i * 32 + 8 * k, k0 + (at + 128 * k), id, i < 2 || k > 0);
                ptx::umma_commit(bar(L::DsFull + (n & 1)));
                ptx::umma_commit(bar(L::VpEmpty + (n & 1)));
                ptx::umma_commit(bar(L::Empty + s));
            }
            __syncwarp();
            if (++s == S) s = 0;
        }
        if (leader) ptx::umma_commit(bar(L::Drain));
        __syncwarp();
        drain_bar(bar(L::Drain), 0);
    } else if (warp == 1) {
        const Source in[2] = {
            {&tm_key, static_cast<const __nv_bfloat16 *>(REV ? p.q : p.k), REV ? p.q_stride : p.k_stride, kh, p.in_k, DK / 64,
             REV ? plan.vec_q : plan.vec_k},
            {&tm_val, static_cast<const __nv_bfloat16 *>(REV ? p.dout : p.v), REV ? (int64_t)p.n_heads * p.in_v : p.v_stride, head,
             p.in_v, p.d_v > 64 ? 2 : 1, REV ? plan.vec_o : plan.vec_v}};
        const TileGates *gates = gates_of(plan.gates, p, sg.seq, (int64_t)sg.index * (plan.seg / C), head);
        int begun = 0;  // tiles whose copies were begun
        for (int n = 0; n < steps; ++n) {
            const int s = n % S, c = tile(n), rows = rows_of(c);
            if (n >= S) wait(L::Empty + s, n / S - 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t at = base + s * L::kStage, m = bar(L::Full + s);
            const int64_t t0 = sg.t0 + (int64_t)c * C;
            const uint32_t bytes = copies ? L::kKey + in[1].halves * kHalf : 0;
            if (!copies) {
                const uint32_t to[2] = {at + L::K, at + L::V};
                tiles_by_threads(in, to, 2, t0, rows, lane, 32);
                rows_loaded();
            } else if (rows < C) {
                // copied whole; what is another sequence's goes before it is handed over
                const uint32_t by = bar(L::Partial);
                if (lane == 0) {
                    ptx::mbar_arrive_tx(by, bytes);
                    tile_by_copy(in[0], at + L::K, t0, by);
                    tile_by_copy(in[1], at + L::V, t0, by);
                }
                if (!wait_bar(by, 0)) drain_bar(by, 0);
                clear_rows(at + L::K, in[0].halves, kHalf, rows, C);
                clear_rows(at + L::V, in[1].halves, kHalf, rows, C);
                ptx::fence_proxy_async();
                __syncwarp();
            }
            if (lane == 0) {
                const bool whole = copies && rows == C;
                ptx::mbar_arrive_tx(m, (uint32_t)sizeof(TileGates) + (whole ? bytes : 0));
                if (whole) {
                    tile_by_copy(in[0], at + L::K, t0, m);
                    tile_by_copy(in[1], at + L::V, t0, m);
                }
                if (n == 0) gdr::wait_for_previous_kernel();  // the gates
                bulk_load(at + L::Gate, gates + (int64_t)c * p.n_heads, sizeof(TileGates), m);
            }
            begun = n + 1;
        }
        // nothing may land in shared memory after the block has gone
        if (!ok)
            for (int n = max(0, begun - S); n < begun; ++n) drain_bar(bar(L::Full + n % S), (n / S) & 1);
    } else if (warp == 2) {
        if (lane == 0) {
            int kept = 0;
            for (int n = 0; n < nc; ++n) {
                if (!enters(n)) continue;
                wait(L::OutFull, kept);
                const int64_t block = block_base(p.cu_seqlens, sg.seq) + ((int64_t)sg.index * (plan.seg / C) + tile(n)) / 2;
                char *to = bp.states + (block * p.n_heads + head) * pair_bytes(DK, DV) + (REV ? 2 * plane_bytes(DK, DV) : 0);
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(base + L::Out),
                             "r"(2 * plane_bytes(DK, DV)) : "memory");
                ptx::bulk_commit();
                ptx::bulk_wait_read0();
                ptx::mbar_arrive(bar(L::OutEmpty));
                ++kept;
            }
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // written, for the next kernel to read
        }
    } else if (warp >= 4 && warp < 8) {
        for (int n = 0; n < steps; ++n) {
            const int s = n % S;
            wait(L::Full + s, n / S);
            auto ready = [&] {
                if (n >= 2) wait(L::VpEmpty + (n & 1), (n >> 1) - 1);
                ptx::tc_fence_after();
            };
            const TileGates *g = reinterpret_cast<const TileGates *>(smem + s * L::kStage + L::Gate);
            if (32 * (warp & 3) < p.d_v)  // other lanes' rows are not read
                scale_values<3>(base + s * L::kStage + L::V, tmem, 256 + (n & 1) * 96, REV ? g->gam : g->del, 1.f, ready);
            else ready();
            ptx::tc_fence_before();
            warp_arrive(bar(L::VpFull + (n & 1)));
            warp_arrive(bar(L::Empty + s));
        }
    } else if (warp >= 8) {
        constexpr int NC = DK / 2;  // key channels of a thread
        const int dv = (warp & 3) * 32 + lane, part = (warp - 8) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const bool live = 32 * (warp & 3) < DV;  // the channels that are kept
        float st[NC];
        const bool cut = sg.index > 0 || !sg.last;
        gdr::wait_for_previous_kernel();
        if (cut) load_state<NC>(st, of_walk<DK>(plan, p, REV).states + ((size_t)slot * p.n_heads + head) * state_floats(DK), dv, part * NC);
        else {
            const float *from = REV ? p.dh_final : p.h0;
            load_given<NC>(st, from ? from + state_at : nullptr, p.d_k, p.d_v, dv, part * NC);
        }
        int kept = 0;
        Factors decays;
#pragma unroll 1
        for (int n = 0; n < nc; ++n) {
            if (enters(n)) {
                if (kept > 0) wait(L::OutEmpty, kept - 1);
                if (live) {
#pragma unroll
                    for (int i = 0; i < NC; i += 8) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) split(st[i + 2 * j], st[i + 2 * j + 1], hi[j], lo[j]);
                        const int c = part * NC + i;
                        const uint32_t at = base + L::Out + (c >> 6) * (DV * 128) + gdr::tile_off<128>(dv, c & 63);
                        gdr::st_shared_16(at, hi);
                        gdr::st_shared_16(at + plane_bytes(DK, DV), lo);
                    }
                }
                ptx::fence_proxy_async();
                warp_arrive(bar(L::OutFull));
                ++kept;
            }
            if (n >= steps) break;
            const int s = n % S;
            wait(L::Full + s, n / S);
            const float whole = decays.next(reinterpret_cast<const TileGates *>(smem + s * L::kStage + L::Gate)->whole);
            warp_arrive(bar(L::Empty + s));
            wait(L::DsFull + (n & 1), n >> 1);
            ptx::tc_fence_after();
            if (32 * (warp & 3) < p.d_v)
#pragma unroll
                for (int i = 0; i < NC; i += 16) {
                    float d[16];
                    ptx::tmem_ld16(lanes + (n & 1) * 128 + part * NC + i, reinterpret_cast<uint32_t *>(d));
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) st[i + j] = fmaf(whole, st[i + j], d[j]);
                }
            ptx::tc_fence_before();
            warp_arrive(bar(L::DsEmpty + (n & 1)));
        }
        if (REV && sg.index == 0 && p.dh0) store_given<NC>(st, p.dh0 + state_at, p.d_k, p.d_v, dv, part * NC);
    }
    __syncwarp();
    __syncthreads();
    if (warp == 0) ptx::tmem_dealloc(tmem, 512);
}

// every segment in reverse and forward, side by side
template <int DK, int DV>
__global__ void __launch_bounds__(kWalkThreads, 1)
    dla_states_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const DlaArgs p,
                      const BwdPlan bp, bool copies) {
    gdr::let_next_kernel_start();
    const unsigned pair = blockIdx.x / (2 * p.n_heads), head = blockIdx.x % p.n_heads, unit = pair * p.n_heads + head;
    if (blockIdx.x / p.n_heads % 2 == 0) state_walk<DK, DV, true>(tm_q, tm_o, p, bp, copies, unit);
    else state_walk<DK, DV, false>(tm_k, tm_v, p, bp, copies, unit);
}

// ---------------------------------------------------------------- gradients
// One unit is a block of 128 tokens and a value head; a CTA takes every gridDim.x-th. Tensor memory, four
// accumulators of 128 columns (rows r: queries, j: keys):
//   T0 = K Q^T (j x r) -> P^T, T1 = V dO^T (j x r) -> W^T, T2 = dO V^T (r x j) -> W as bf16 planes in their
//   place: 16 columns become a step's 8 + 8;  T3 = dO S0^T -> times scale gamma_r -> + W K = dQ
//   then T2 = K dS1, T3 = V dS1^T -> times delta_j -> + P^T dO = dV, + W^T Q = dK
// W is formed in both orders of rows, because an A operand in tensor memory has its rows in the lanes.
// warps: 0 issues products, 1 loads tiles, 2 loads states, 3 gates and dg, 4..7 <S0, dS1>, 8..15 the rows r,
// 16..23 the rows j (two warps a quarter of the lanes, half the columns each)
constexpr int kGradThreads = 768;
// Registers a thread has at launch, and those of the warps that serve and of the rows' after they gave away
// or took some: together what the block was launched with.
constexpr int kGradRegs = 80, kGradServe = 48, kGradRows = 96;
static_assert(8 * kGradServe + 16 * kGradRows == 24 * kGradRegs, "the launch's registers");

struct BlockGates {
    float2 G[kBlock];
    float gam[kBlock], del[kBlock];  // gam: times scale
    float whole, pad[3];
};
// what dg is summed from
struct BlockSums {
    float a[2][kBlock], b[2][kBlock], col[2][kBlock], row[4][kBlock], ss[4];
};

template <int DK, int DV>
struct GradSmem {
    static constexpr int kKey = DK / 64 * kWide, kVal = DV / 64 * kWide, kPlane = plane_bytes(DK, DV);
    static constexpr int Q = 0, K = kKey, V = 2 * kKey, dO = V + kVal, X = dO + kVal, Gate = X + 2 * kPlane;
    static constexpr int Sums = Gate + 2 * (int)sizeof(BlockGates), Bars = Sums + (int)sizeof(BlockSums);
    static constexpr int KqFull = 0, VoFull = 1, KvEmpty = 2, X0Full = 3, X1Full = 4, X0Empty = 5, X1Empty = 6, F1 = 7, F2 = 8,
                         WFull = 9, F3 = 10, AEmpty = 11, F4 = 12, PFull = 13, Scaled = 14, F5 = 15, CEmpty = 16, GFull = 17,
                         GEmpty = 19, SumsFull = 21, SumsEmpty = 22, Drain = 23, Partial = 24, QoEmpty = 26, F2w = 27, CvEmpty = 28, kBars = 30;
    static constexpr int kBytes = Bars + 8 * kBars + 16 + 1024;  // the base is rounded up to 1024
    static_assert(sizeof(BlockGates) % 16 == 0 && sizeof(BlockSums) % 16 == 0 && kBytes <= 227 * 1024, "fits an SM");
};

struct Block {
    int seq, head, len;  // len = 0: an unused slot
    int64_t slot, t0, index;
};
__device__ __forceinline__ Block find_block(const DlaArgs &p, int64_t unit) {
    Block b;
    b.head = (int)(unit % p.n_heads);
    b.slot = unit / p.n_heads;
    int lo = 0, hi = p.n_seq - 1;  // largest n with block_base(n) <= slot
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (block_base(p.cu_seqlens, mid) <= b.slot) lo = mid; else hi = mid - 1;
    }
    b.seq = lo;
    b.index = b.slot - block_base(p.cu_seqlens, lo);
    b.t0 = p.cu_seqlens[lo] + b.index * kBlock;
    const int64_t left = p.cu_seqlens[lo + 1] - b.t0;
    b.len = left < 0 ? 0 : left < kBlock ? (int)left : kBlock;
    return b;
}

// 128 rows of a tile by a tensor copy of 64 channels x 128 tokens, or by a warp
__device__ __forceinline__ void wide_tile(const Source &s, uint32_t dst, int64_t t0, int rows, int lane) {
    const __nv_bfloat16 *p = s.base + t0 * s.stride + (int64_t)s.head * s.d;
#pragma unroll 1
    for (int h = 0; h < s.halves; ++h)
#pragma unroll 1
        for (int r = 0; r < kBlock; r += C)
            gdr::load_tile<__nv_bfloat16, 128>(dst + h * kWide + r * 128, 0, p + (rows > r ? r * s.stride : 0) + h * 64, s.stride, rows - r,
                                               s.d - h * 64, s.vec, lane, 32);
}

// N channels from c0 on of a row, to bf16 or fp32
template <int N>
__device__ __forceinline__ void store_row(__nv_bfloat16 *to, const float *x, int c0, int d, int wide) {
#pragma unroll
    for (int i = 0; i < N; i += 16) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = ptx::pack_bf16(x[i + 2 * j], x[i + 2 * j + 1]);
        const int c = c0 + i;
        if (wide == 2) {
            if (c < d)
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to + c), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                             "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
        } else if (wide == 1) {
            if (c < d) *reinterpret_cast<uint4 *>(to + c) = make_uint4(w[0], w[1], w[2], w[3]);
            if (c + 8 < d) *reinterpret_cast<uint4 *>(to + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < d) reinterpret_cast<uint16_t *>(to)[c + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
    }
}
template <int N>
__device__ __forceinline__ void store_part(float *to, const float *x) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(to + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}

// sixteen values of each lane summed over the warp's lanes: the sum of value i to the lanes 2 i and 2 i + 1
__device__ __forceinline__ float sum_over_lanes(float *v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16, n = 8; n > 0; o >>= 1, n >>= 1)
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float keep = lane & o ? v[k + n] : v[k], give = lane & o ? v[k] : v[k + n];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

template <int DK, int DV>
__global__ void __launch_bounds__(kGradThreads, 1)
    dla_grad_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const DlaArgs p,
                    const BwdPlan bp, bool copies, int wide_k, int wide_v, int64_t units) {
    using L = GradSmem<DK, DV>;
    extern __shared__ __align__(1024) char smem_raw[];
    char *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };  // equal over a warp, and told so
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int group = p.n_heads / p.n_k_heads;
    auto bar = [&](int i) { return base + L::Bars + 8 * i; };
    BlockGates *gates = reinterpret_cast<BlockGates *>(smem + L::Gate);
    BlockSums &sums = *reinterpret_cast<BlockSums *>(smem + L::Sums);
    if (tid == 0) {
        const int ones[] = {L::KqFull, L::VoFull, L::X0Full, L::X1Full, L::X0Empty, L::F1, L::F2w, L::F2, L::F3, L::F4, L::F5, L::GFull,
                            L::GFull + 1, L::SumsEmpty, L::Drain, L::Partial, L::Partial + 1};
        for (int i : ones) ptx::mbar_init(bar(i), 1);
        const int eights[] = {L::WFull, L::AEmpty, L::PFull, L::Scaled, L::CvEmpty, L::CEmpty};
        for (int i : eights) ptx::mbar_init(bar(i), 8);
        ptx::mbar_init(bar(L::KvEmpty), 1 + 8);  // the products, the rows' warps that read it
        ptx::mbar_init(bar(L::QoEmpty), 1 + 8);
        ptx::mbar_init(bar(L::X1Empty), 1 + 4);
        ptx::mbar_init(bar(L::GEmpty), 16 + (p.dg ? 1 : 0));
        ptx::mbar_init(bar(L::GEmpty + 1), 16 + (p.dg ? 1 : 0));
        ptx::mbar_init(bar(L::SumsFull), 16 + 4);
        ptx::mbar_init_fence();
    }
    if (warp == 0) ptx::tmem_alloc(bar(L::kBars), 512);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<const uint32_t *>(smem + L::Bars + 8 * L::kBars);
    constexpr uint32_t T0 = 0, T1 = 128, T2 = 256, T3 = 384;
    bool ok = true;
    auto wait = [&](int b, int parity) { ok = wait_bar(bar(b), parity & 1) && ok; };
    gdr::wait_for_previous_kernel();
    int i = 0;  // units so far
    // the roles walk over the same units
    auto next_unit = [&](int64_t &u, Block &b) {
        for (; u < units; u += gridDim.x) {
            b = find_block(p, u);
            if (uniform(b.len) > 0) return true;
        }
        return false;
    };
    Block b;

    if (warp == 0) {
        ptx::regs_decrease<kGradServe>();
        const uint32_t leader = ptx::elect_one();
        constexpr uint32_t id_pair = ptx::idesc_bf16(128, 128, 0, 0), id_k = ptx::idesc_bf16(128, DK, 0, 1);
        constexpr uint32_t id_v = ptx::idesc_bf16(128, DV, 0, 1), id_vk = ptx::idesc_bf16(128, DV, 0, 0);
        auto rows = [&](int tile) { return ptx::sdesc_sw128(base + tile, 16, 1024); };         // K-major, 16 channels a step
        auto cols = [&](int tile, int part) { return ptx::sdesc_sw128(base + tile, part, 1024); };  // MN-major, 16 rows a step
        auto step = [](int k) { return (uint32_t)((k >> 2) * kWide + (k & 3) * 32) / 16; };
        auto plane_step = [](int k) { return (uint32_t)((k >> 2) * (DV * 128) + (k & 3) * 32) / 16; };
        const uint64_t q = rows(L::Q), k = rows(L::K), v = rows(L::V), o = rows(L::dO), x = rows(L::X);
        const uint64_t qc = cols(L::Q, kWide), kc = cols(L::K, kWide), oc = cols(L::dO, kWide), xc = cols(L::X, DV * 128);
        for (int64_t u = blockIdx.x; next_unit(u, b); u += gridDim.x, ++i) {
            wait(L::KqFull, i);
            ptx::tc_fence_after();
            if (leader) {
#pragma unroll
                for (int n = 0; n < DK / 16; ++n) ptx::umma_ss(tmem + T0, k + step(n), q + step(n), id_pair, n > 0);
            }
            __syncwarp();
            wait(L::VoFull, i);
            if (leader) {
#pragma unroll
                for (int n = 0; n < DV / 16; ++n) ptx::umma_ss(tmem + T1, v + step(n), o + step(n), id_pair, n > 0);
                ptx::umma_commit(bar(L::F1));
            }
            __syncwarp();
            if (i > 0) wait(L::CvEmpty, i - 1);
            ptx::tc_fence_after();
            if (leader) {
#pragma unroll
                for (int n = 0; n < DV / 16; ++n) ptx::umma_ss(tmem + T2, o + step(n), v + step(n), id_pair, n > 0);
                ptx::umma_commit(bar(L::F2w));
            }
            __syncwarp();
            wait(L::X0Full, i);
            if (i > 0) wait(L::CEmpty, i - 1);
            ptx::tc_fence_after();
            if (leader) {
#pragma unroll
                for (int h = 1; h >= 0; --h)  // the small plane first
#pragma unroll
                    for (int n = 0; n < DV / 16; ++n)
                        ptx::umma_ss(tmem + T3, o + step(n), xc + (uint32_t)(h * L::kPlane / 16 + 128 * n), id_k, h == 0 || n > 0);
                ptx::umma_commit(bar(L::F2));
                ptx::umma_commit(bar(L::X0Empty));
            }
            __syncwarp();
            wait(L::WFull, i);
            ptx::tc_fence_after();
            if (leader) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < kBlock / 16; ++n)
                        ptx::umma_ts(tmem + T3, tmem + T2 + 16 * n + 8 * h, kc + (uint32_t)(128 * n), id_k, 1);
                ptx::umma_commit(bar(L::F3));
            }
            __syncwarp();
            wait(L::X1Full, i);
            wait(L::F3, i);  // W is read; dQ leaves tensor memory beside the next product
            ptx::tc_fence_after();
            if (leader) {
#pragma unroll
                for (int h = 1; h >= 0; --h)  // the small plane first
#pragma unroll
                    for (int n = 0; n < DK / 16; ++n)
                        ptx::umma_ss(tmem + T2, k + step(n), x + (uint32_t)(h * L::kPlane / 16) + plane_step(n), id_vk, h == 0 || n > 0);
            }
            __syncwarp();
            wait(L::AEmpty, i);
            ptx::tc_fence_after();
            if (leader) {
#pragma unroll
                for (int h = 1; h >= 0; --h)  // the small plane first
#pragma unroll
                    for (int n = 0; n < DV / 16; ++n)
                        ptx::umma_ss(tmem + T3, v + step(n), xc + (uint32_t)(h * L::kPlane / 16 + 128 * n), id_k, h == 0 || n > 0);
                ptx::umma_commit(bar(L::F4));
                ptx::umma_commit(bar(L::X1Empty));
                ptx::umma_commit(bar(L::KvEmpty));
            }
            __syncwarp();
            wait(L::PFull, i);
            wait(L::Scaled, i);
            ptx::tc_fence_after();
            if (leader) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < kBlock / 16; ++n)
                        ptx::umma_ts(tmem + T2, tmem + T0 + 16 * n + 8 * h, oc + (uint32_t)(128 * n), id_v, 1);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < kBlock / 16; ++n)
                        ptx::umma_ts(tmem + T3, tmem + T1 + 16 * n + 8 * h, qc + (uint32_t)(128 * n), id_k, 1);
                ptx::umma_commit(bar(L::F5));
                ptx::umma_commit(bar(L::QoEmpty));
            }
            __syncwarp();
        }
        if (leader) ptx::umma_commit(bar(L::Drain));
        __syncwarp();
        drain_bar(bar(L::Drain), 0);
    } else if (warp == 1) {
        ptx::regs_decrease<kGradServe>();
        int partials = 0;
        for (int64_t u = blockIdx.x; next_unit(u, b); u += gridDim.x, ++i) {
            if (i > 0) wait(L::KvEmpty, i - 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // Keys and values are free two products before queries and dO: half of the next unit's copies begin
            // then (two sequences of 8K tokens, 32 heads: 573 us with all of them at the end, 545 so). The copies are
            // written out: from an array of their sources, walked by a loop, they began 2 us a unit later.
            const int kh = b.head / group;
            const bool whole = b.len == kBlock;
            auto copy = [&](const CUtensorMap &map, int to, int halves, int head, uint32_t m) {
                for (int h = 0; h < halves; ++h) ptx::tma_load_3d(base + to + h * kWide, &map, h * 64, head, (int)b.t0, m);
            };
            if (copies) {
                // a partial block is copied whole; what is another sequence's goes before it is handed over
                const uint32_t kq = bar(whole ? L::KqFull : L::Partial), vo = bar(whole ? L::VoFull : L::Partial + 1);
                if (lane == 0) {
                    ptx::mbar_arrive_tx(kq, 2 * L::kKey);
                    copy(tm_k, L::K, DK / 64, kh, kq);
                    ptx::mbar_arrive_tx(vo, 2 * L::kVal);
                    copy(tm_v, L::V, DV / 64, b.head, vo);
                }
                if (i > 0) wait(L::QoEmpty, i - 1);  // given up: the copies come all the same, to be waited for
                if (lane == 0) {
                    copy(tm_q, L::Q, DK / 64, kh, kq);
                    copy(tm_o, L::dO, DV / 64, b.head, vo);
                }
                if (!whole) {
                    if (!wait_bar(kq, partials & 1)) drain_bar(kq, partials & 1);
                    clear_rows(base + L::K, DK / 64, kWide, b.len, kBlock);
                    clear_rows(base + L::Q, DK / 64, kWide, b.len, kBlock);
                    ptx::fence_proxy_async();
                    warp_arrive(bar(L::KqFull));
                    if (!wait_bar(vo, partials & 1)) drain_bar(vo, partials & 1);
                    clear_rows(base + L::V, DV / 64, kWide, b.len, kBlock);
                    clear_rows(base + L::dO, DV / 64, kWide, b.len, kBlock);
                    ptx::fence_proxy_async();
                    warp_arrive(bar(L::VoFull));
                    ++partials;
                }
            } else {
                const int64_t ov = (int64_t)p.n_heads * p.in_v;
                const Source in[4] = {{&tm_k, static_cast<const __nv_bfloat16 *>(p.k), p.k_stride, kh, p.in_k, DK / 64, bp.walk.vec_k},
                                      {&tm_v, static_cast<const __nv_bfloat16 *>(p.v), p.v_stride, b.head, p.in_v, DV / 64, bp.walk.vec_v},
                                      {&tm_q, static_cast<const __nv_bfloat16 *>(p.q), p.q_stride, kh, p.in_k, DK / 64, bp.walk.vec_q},
                                      {&tm_o, static_cast<const __nv_bfloat16 *>(p.dout), ov, b.head, p.in_v, DV / 64, bp.walk.vec_o}};
                const int to[4] = {L::K, L::V, L::Q, L::dO};
                if (i > 0) wait(L::QoEmpty, i - 1);
#pragma unroll 1
                for (int n = 0; n < 4; ++n) wide_tile(in[n], base + to[n], b.t0, b.len, lane);
                rows_loaded();
                if (lane == 0) {
                    ptx::mbar_arrive(bar(L::KqFull));
                    ptx::mbar_arrive(bar(L::VoFull));
                }
            }
        }
        // nothing may land in shared memory after the block has gone
        if (!ok && i > 0) {
            drain_bar(bar(L::KqFull), (i - 1) & 1);
            drain_bar(bar(L::VoFull), (i - 1) & 1);
        }
    } else if (warp == 2) {
        ptx::regs_decrease<kGradServe>();
        if (lane == 0) {
            for (int64_t u = blockIdx.x; ; u += gridDim.x, ++i) {
                bool more = false;
                for (; u < units; u += gridDim.x) {
                    b = find_block(p, u);
                    if (b.len > 0) {
                        more = true;
                        break;
                    }
                }
                if (!more) break;
                const char *from = bp.states + (b.slot * p.n_heads + b.head) * pair_bytes(DK, DV);
                if (i > 0) wait(L::X1Empty, i - 1);
                if (!ok) break;
                ptx::mbar_arrive_tx(bar(L::X0Full), 2 * L::kPlane);
                bulk_load(base + L::X, from, 2 * L::kPlane, bar(L::X0Full));
                wait(L::X0Empty, i);
                if (!ok) {
                    drain_bar(bar(L::X0Full), i & 1);
                    break;
                }
                ptx::mbar_arrive_tx(bar(L::X1Full), 2 * L::kPlane);
                bulk_load(base + L::X, from + 2 * L::kPlane, 2 * L::kPlane, bar(L::X1Full));
            }
            if (!ok && i > 0) drain_bar(bar(L::X1Full), (i - 1) & 1);
        }
        __syncwarp();
    } else if (warp == 3) {
        ptx::regs_decrease<kGradServe>();
        // gates: four tokens a lane, of two tiles' sums
        auto form = [&](const Block &c, int n) {
            BlockGates &g = gates[n & 1];
            if (n >= 2) wait(L::GEmpty + (n & 1), (n >> 1) - 1);
            const TileGates *t = gates_of(bp.walk.gates, p, c.seq, 2 * c.index, c.head);
            const bool two = c.len > C;
            float2 s0 = from_fixed(t->sum), s1 = make_float2(0.f, 0.f);
            s0.x += nan_of(*t);
            if (two) {
                s1 = from_fixed(t[p.n_heads].sum);
                s1.x += nan_of(t[p.n_heads]);
            }
            const Two total = add({s0.x, s0.y}, {s1.x, s1.y});
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
                const int r = lane + 32 * e;
                Two G = total;
                if (r < C) G = {t->G[r].x, t->G[r].y};
                else if (two) G = add({s0.x, s0.y}, {t[p.n_heads].G[r - C].x, t[p.n_heads].G[r - C].y});
                g.G[r] = make_float2(G.hi, G.lo);
                g.gam[r] = p.scale * ex2(G.hi) * ex2(G.lo);  // a whole part and a fraction, or a sum of such
                g.del[r] = exp2_between(make_float2(total.hi, total.lo), make_float2(G.hi, G.lo));
            }
            if (lane == 0) g.whole = ex2(total.hi) * ex2(total.lo);
            warp_arrive(bar(L::GFull + (n & 1)));
        };
        auto decays = [&](const Block &c, int n) {  // dg of a unit, four neighbouring tokens a lane
            wait(L::SumsFull, n);
            const float whole = gates[n & 1].whole * ((sums.ss[0] + sums.ss[1]) + (sums.ss[2] + sums.ss[3]));
            Two a[4], v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 4 * lane + e;
                float row = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (w <= r >> 5) row += sums.row[w][r];
                const float col = sums.col[0][r] + sums.col[1][r];
                a[e] = add({sums.a[0][r] + sums.a[1][r], 0.f}, add({row, 0.f}, {-col, 0.f}));
                v[e] = {sums.b[0][r] + sums.b[1][r], 0.f};
            }
            warp_arrive(bar(L::SumsEmpty));
            warp_arrive(bar(L::GEmpty + (n & 1)));
            const Two sa = warp_scan(add(add(a[0], a[1]), add(a[2], a[3]))), sb = warp_scan(add(add(v[0], v[1]), add(v[2], v[3])));
            const Two total = last_lane(sa);
            Two a0 = up(sa, 1), b0 = up(sb, 1);
            if (lane == 0) a0 = b0 = {0.f, 0.f};
            float both = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 4 * lane + e;
                const Two sum = add(minus(total, a0), add({whole, 0.f}, b0));
                if (r < c.len) {  // nothing passes a decay of 0: what the sums leave there is rounding
                    const float d = p.g[(c.t0 + r) * p.g_stride + c.head] < kGFloor ? 0.f : sum.hi + sum.lo;
                    if (p.g_stride == 0) both += d;
                    else p.dg[(c.t0 + r) * p.n_heads + c.head] = d;
                }
                a0 = add(a0, a[e]);
                b0 = add(b0, v[e]);
            }
            if (p.g_stride == 0) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) both += __shfl_xor_sync(0xffffffffu, both, o);
                if (lane == 0) bp.sums[c.slot * p.n_heads + c.head] = both;
            }
        };
        if (p.dg && p.g_stride == 0)  // unused slots count nothing
            for (int64_t u = blockIdx.x; u < units; u += gridDim.x)
                if (find_block(p, u).len == 0 && lane == 0) bp.sums[u] = 0.f;
        Block last{};
        for (int64_t u = blockIdx.x; next_unit(u, b); u += gridDim.x, ++i) {
            form(b, i);
            if (i > 0 && p.dg) decays(last, i - 1);
            last = b;
        }
        if (i > 0 && p.dg) decays(last, i - 1);
    } else if (warp < 8) {
        ptx::regs_decrease<kGradServe>();
        // <S0, dS1>: dS1 from shared memory, S0, which was there before it, from L2
        const int t = tid - 128;
        for (int64_t u = blockIdx.x; next_unit(u, b); u += gridDim.x, ++i) {
            wait(L::X1Full, i);
            float ss = 0.f;
            if (p.dg) {
                const char *from = bp.states + (b.slot * p.n_heads + b.head) * pair_bytes(DK, DV);
#pragma unroll 2
                for (int n = t; n < L::kPlane / 16; n += 128) {
                    const uint4 h0 = reinterpret_cast<const uint4 *>(from)[n], l0 = reinterpret_cast<const uint4 *>(from + L::kPlane)[n];
                    const uint4 h1 = reinterpret_cast<const uint4 *>(smem + L::X)[n], l1 = reinterpret_cast<const uint4 *>(smem + L::X + L::kPlane)[n];
                    const uint32_t x[4] = {h0.x, h0.y, h0.z, h0.w}, y[4] = {l0.x, l0.y, l0.z, l0.w};
                    const uint32_t z[4] = {h1.x, h1.y, h1.z, h1.w}, w[4] = {l1.x, l1.y, l1.z, l1.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        ss = fmaf(gdr::lo_f(x[e]) + gdr::lo_f(y[e]), gdr::lo_f(z[e]) + gdr::lo_f(w[e]), ss);
                        ss = fmaf(gdr::hi_f(x[e]) + gdr::hi_f(y[e]), gdr::hi_f(z[e]) + gdr::hi_f(w[e]), ss);
                    }
                }
            }
            warp_arrive(bar(L::X1Empty));
            if (p.dg) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (i > 0) wait(L::SumsEmpty, i - 1);
                if (lane == 0) sums.ss[warp - 4] = ss;
                warp_arrive(bar(L::SumsFull));
            }
        }
    } else {
        ptx::regs_increase<kGradRows>();
        // the rows r (queries: W, dQ) and the rows j (keys: P^T, W^T, dV, dK)
        const bool keys = warp >= 16;
        const int w = warp & 3, part = (warp >> 2) & 1, x = 32 * w + lane;  // this thread's row
        const uint32_t lanes = tmem + ((uint32_t)(w * 32) << 16);
        constexpr int NK = DK / 2, NV = DV / 2;  // a part's columns
        for (int64_t u = blockIdx.x; next_unit(u, b); u += gridDim.x, ++i) {
            wait(L::GFull + (i & 1), i >> 1);
            const BlockGates &g = gates[i & 1];
            const float2 G = g.G[x];
            wait(keys ? L::F1 : L::F2w, i);
            ptx::tc_fence_after();
            if (p.dg && i > 0) wait(L::SumsEmpty, i - 1);
            float col = 0.f;
            // blocks of 32 columns, two a part, so that both parts have as many below the diagonal
#pragma unroll 1
            for (int n = 0; n < 4; ++n) {
                const int B = n < 2 ? (part ? 1 : 0) : (part ? 2 : 3), c0 = 32 * B + 16 * (n & 1);
                const uint32_t at = lanes + c0;
                if (keys ? B < w : B > w) {  // above the diagonal
                    uint32_t zero[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) zero[e] = 0;
                    if (keys) ptx::tmem_st16(at + T0, zero);
                    ptx::tmem_st16(at + (keys ? T1 : T2), zero);
                    continue;
                }
                float ov[16], kq[16];
                ptx::tmem_ld16(at + (keys ? T1 : T2), reinterpret_cast<uint32_t *>(ov));
                if (keys) ptx::tmem_ld16(at + T0, reinterpret_cast<uint32_t *>(kq));
                ptx::tmem_ld_wait();
                uint32_t pl[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const int c = c0 + e;
                    const float4 Gc = *reinterpret_cast<const float4 *>(&g.G[c]);
                    const float2 Ga = make_float2(Gc.x, Gc.y), Gb = make_float2(Gc.z, Gc.w);
                    float ea, eb;
                    if (keys) {
                        ea = c >= x ? p.scale * exp2_between(Ga, G) : 0.f;
                        eb = c + 1 >= x ? p.scale * exp2_between(Gb, G) : 0.f;
                        // what is masked may be anything, a NaN of another token's too
                        split(c >= x ? ea * kq[e] : 0.f, c + 1 >= x ? eb * kq[e + 1] : 0.f, pl[e >> 1], pl[8 + (e >> 1)]);
                        ov[e] = c >= x ? ea * ov[e] : 0.f;
                        ov[e + 1] = c + 1 >= x ? eb * ov[e + 1] : 0.f;
                        kq[e] = c > x ? ov[e] * kq[e] : 0.f;
                        kq[e + 1] = c + 1 > x ? ov[e + 1] * kq[e + 1] : 0.f;
                        col += kq[e] + kq[e + 1];
                    } else {
                        ov[e] = c <= x ? p.scale * exp2_between(G, Ga) * ov[e] : 0.f;
                        ov[e + 1] = c + 1 <= x ? p.scale * exp2_between(G, Gb) * ov[e + 1] : 0.f;
                    }
                }
                if (keys) {
                    ptx::tmem_st16(at + T0, pl);
                    if (p.dg) {
                        const float row = sum_over_lanes(kq);
                        if ((lane & 1) == 0) sums.row[w][c0 + (lane >> 1)] = row;
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; e += 2) split(ov[e], ov[e + 1], pl[e >> 1], pl[8 + (e >> 1)]);
                ptx::tmem_st16(at + (keys ? T1 : T2), pl);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            // the part of the state: times gamma or delta, and its dot product with the row's q or k
            const float f = keys ? g.del[x] : g.gam[x];
            if (keys) warp_arrive(bar(L::PFull));
            wait(keys ? L::F4 : L::F2, i);
            ptx::tc_fence_after();
            float dot = 0.f;
#pragma unroll 1
            for (int c = part * NK; c < (part + 1) * NK; c += 16) {
                float y[16];
                ptx::tmem_ld16(lanes + T3 + c, reinterpret_cast<uint32_t *>(y));
                ptx::tmem_ld_wait();
                if (p.dg) {
#pragma unroll
                    for (int e = 0; e < 16; e += 8) {
                        const uint4 t = *reinterpret_cast<const uint4 *>(smem + (keys ? L::K : L::Q) + ((c + e) >> 6) * kWide +
                                                                         gdr::tile_off<128>(x, (c + e) & 63));
                        const uint32_t z[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            dot = fmaf(gdr::lo_f(z[j]), y[e + 2 * j], dot);
                            dot = fmaf(gdr::hi_f(z[j]), y[e + 2 * j + 1], dot);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] *= f;
                ptx::tmem_st16(lanes + T3 + c, reinterpret_cast<const uint32_t *>(y));
            }
            if (keys)
#pragma unroll 1
                for (int c = part * NV; c < (part + 1) * NV; c += 16) {
                    float y[16];
                    ptx::tmem_ld16(lanes + T2 + c, reinterpret_cast<uint32_t *>(y));
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] *= f;
                    ptx::tmem_st16(lanes + T2 + c, reinterpret_cast<const uint32_t *>(y));
                }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            warp_arrive(bar(keys ? L::Scaled : L::WFull));
            warp_arrive(bar(L::GEmpty + (i & 1)));
            warp_arrive(bar(keys ? L::KvEmpty : L::QoEmpty));
            if (p.dg) {
                if (keys) {
                    sums.b[part][x] = f * dot;
                    sums.col[part][x] = col;
                } else {
                    sums.a[part][x] = f * dot;
                }
                warp_arrive(bar(L::SumsFull));
            }
            // the results
            wait(keys ? L::F5 : L::F3, i);
            ptx::tc_fence_after();
            const int64_t t = b.t0 + x;
            const bool in = x < b.len;
            if (keys) {
                __nv_bfloat16 *dv = static_cast<__nv_bfloat16 *>(p.dv) + (t * p.n_heads + b.head) * p.d_v;
#pragma unroll 1
                for (int c = part * NV; c < (part + 1) * NV; c += 32) {
                    float y[32];
                    ptx::tmem_ld32(lanes + T2 + c, reinterpret_cast<uint32_t *>(y));
                    ptx::tmem_ld_wait();
                    if (in) store_row<32>(dv, y, c, p.d_v, wide_v);
                }
                // the next block's pair product goes there
                ptx::tc_fence_before();
                warp_arrive(bar(L::CvEmpty));
            }
            __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(keys ? p.dk : p.dq) + (t * p.n_k_heads + b.head) * p.d_k;
            float *partial = group > 1 ? (keys ? bp.dk : bp.dq) + (t * p.n_heads + b.head) * DK : nullptr;
#pragma unroll 1
            for (int c = part * NK; c < (part + 1) * NK; c += 32) {
                float y[32];
                ptx::tmem_ld32(lanes + T3 + c, reinterpret_cast<uint32_t *>(y));
                ptx::tmem_ld_wait();
                if (in) {
                    if (partial) store_part<32>(partial + c, y);
                    else store_row<32>(to, y, c, p.d_k, wide_k);
                }
            }
            ptx::tc_fence_before();
            warp_arrive(bar(keys ? L::CEmpty : L::AEmpty));
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 0) ptx::tmem_dealloc(tmem, 512);
}

// dq or dk of a key head: the sum of its value heads' parts, eight channels a thread
template <int DK>
__global__ void __launch_bounds__(256) dla_shared_heads_kernel(const float *dq, const float *dk, const DlaArgs p, bool wide) {
    gdr::wait_for_previous_kernel();
    const int group = p.n_heads / p.n_k_heads;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, rows = p.n_tok * p.n_k_heads;
    const int64_t row = i / (DK / 8);  // token and key head
    const int c = (int)(i % (DK / 8)) * 8;
    if (row >= 2 * rows || c >= p.d_k) return;
    if ((row >= rows ? row - rows : row) / p.n_k_heads >= p.cu_seqlens[p.n_seq]) return;  // behind the last sequence
    const bool second = row >= rows;
    const float *from = (second ? dk : dq) + (second ? row - rows : row) * group * DK + c;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    for (int h = 0; h < group; ++h, from += DK) {
        const float4 a = *reinterpret_cast<const float4 *>(from), b = *reinterpret_cast<const float4 *>(from + 4);
        x[0] += a.x; x[1] += a.y; x[2] += a.z; x[3] += a.w;
        x[4] += b.x; x[5] += b.y; x[6] += b.z; x[7] += b.w;
    }
    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(second ? p.dk : p.dq) + (second ? row - rows : row) * p.d_k + c;
    if (wide) {
        *reinterpret_cast<uint4 *>(to) = make_uint4(ptx::pack_bf16(x[0], x[1]), ptx::pack_bf16(x[2], x[3]),
                                                    ptx::pack_bf16(x[4], x[5]), ptx::pack_bf16(x[6], x[7]));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < p.d_k) to[e] = __float2bfloat16_rn(x[e]);
    }
}

// ---------------------------------------------------------------- host
// Both walks of every sequence and head are a CTA each. Where there are fewer than 96, sequences of more than 16 tiles
// are cut, which costs K, V, Q and dO read once more and the join; the lengths, which would tell more, are on the
// device. Measured both ways, us, heads of 128 channels, cut / whole. Ragged batches of few heads gain: 8K tokens
// with 15 x 512, 8 heads (256 walks, whole) 207 / 254; 64K with 100, 24 heads (96 walks, whole) 1759 / 1973; 16K
// with 100 tokens 496 / 536. Equal lengths of many heads lose: 2 x 8K tokens, 32 heads (128 walks, whole) 649 / 541; one
// of 16K, 48 heads (96, whole) 894 / 796, 47 heads (94, cut) 877 / 782, 32 heads (64, cut) 624 / 611; 4 x 4K,
// 8 heads (64, cut) 199 / 184. The limit of 96 lies between what few long and what many equal ones ask for.
int walk_segment(int64_t n_tok, int32_t n_seq, int32_t n_heads) {
    const int64_t tiles = (n_tok + C - 1) / C;
    if ((int64_t)n_seq * n_heads * 2 >= 96 || tiles <= 16) return (int)std::min<int64_t>((tiles + 1) / 2 * 2, (int64_t)1 << 24) * C;
    // even, so that blocks do not straddle segments
    const int m = segment_tiles(n_tok, n_seq, 2 * n_heads);
    return (m + (m & 1)) * C;
}
struct Layout {
    size_t gates, joins, states, sums, parts, copies, bytes;
    int seg;
    int64_t slots;
};
Layout layout(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k, int32_t d_v) {
    const int dkp = d_k <= 64 ? 64 : 128, dvp = d_v <= 64 ? 64 : 128;
    auto up = [](size_t x) { return (x + 1023) / 1024 * 1024; };
    Layout l;
    l.seg = walk_segment(n_tok, n_seq, n_heads);
    l.slots = n_tok / l.seg + n_seq;
    const size_t units = n_tok > l.seg ? (size_t)l.slots * n_heads : 0, blocks = (size_t)block_slots(n_tok, n_seq) * n_heads;
    l.gates = 0;
    l.joins = up(gate_bytes(n_tok, n_seq, n_heads));
    l.states = l.joins + up(2 * units * (state_floats(dkp) * 4 + sizeof(Two)));
    l.sums = l.states + blocks * pair_bytes(dkp, dvp);
    l.parts = up(l.sums + blocks * 4);
    l.copies = up(l.parts + (n_heads > n_k_heads ? 2 * (size_t)n_tok * n_heads * dkp * 4 : 0));
    l.bytes = l.copies + copies_bytes(n_tok, n_heads, n_k_heads, d_k, d_v, true);
    return l;
}

template <int DK, int DV>
cudaError_t backward(const DlaArgs &args, cudaStream_t stream) {
    DlaArgs p = args;
    const Layout l = layout(p.n_tok, p.n_seq, p.n_heads, p.n_k_heads, p.d_k, p.d_v);
    char *ws = static_cast<char *>(p.workspace);
    cudaError_t e = align_inputs(p, ws + l.copies, true, stream);
    if (e != cudaSuccess) return e;
    BwdPlan bp{};
    Plan &plan = bp.walk;
    plan = make_plan(p, true);
    plan.seg = l.seg;
    plan.slots = l.slots;
    plan.cut = p.n_tok > l.seg;
    plan.states = reinterpret_cast<float *>(ws + l.joins);
    const size_t units = plan.cut ? (size_t)l.slots * p.n_heads : 0;
    plan.decays = reinterpret_cast<Two *>(plan.states + 2 * units * state_floats(DK));
    bp.states = ws + l.states;
    bp.sums = reinterpret_cast<float *>(ws + l.sums);
    bp.dq = reinterpret_cast<float *>(ws + l.parts);
    bp.dk = bp.dq + (size_t)p.n_tok * p.n_heads * DK;
    const int64_t os = (int64_t)p.n_heads * p.in_v;
    CUtensorMap m[4], wm[4];  // q, k, v, dout; tiles of 64 and of 128 tokens
    bool copies = true;
    for (int rows : {C, kBlock}) {
        CUtensorMap *to = rows == C ? m : wm;
        copies = copies && TileMap::encode(&to[0], p.q, p.n_tok, p.q_stride, p.n_k_heads, p.in_k, rows) &&
                 TileMap::encode(&to[1], p.k, p.n_tok, p.k_stride, p.n_k_heads, p.in_k, rows) &&
                 TileMap::encode(&to[2], p.v, p.n_tok, p.v_stride, p.n_heads, p.in_v, rows) &&
                 TileMap::encode(&to[3], p.dout, p.n_tok, os, p.n_heads, p.in_v, rows);
    }
    e = launch_gates(p, plan, stream);
    if (e != cudaSuccess) return e;
    if (plan.cut) {
        e = launch_segments<DK>(p, plan, m[0], m[1], m[2], m[3], copies, 2, stream);
        if (e != cudaSuccess) return e;
    }
    e = gdr::launch_dependent(dla_states_kernel<DK, DV>, dim3((unsigned)(2 * plan.slots * p.n_heads)), kWalkThreads,
                              WalkSmem<DK, DV>::kBytes, stream, m[0], m[1], m[2], m[3], p, bp, copies);
    if (e != cudaSuccess) return e;
    auto wide = [](const void *a, const void *b, int d) {
        const uintptr_t x = (uintptr_t)a | (uintptr_t)b;
        return d % 16 == 0 && x % 32 == 0 ? 2 : d % 8 == 0 && x % 16 == 0 ? 1 : 0;
    };
    const int64_t n = block_slots(p.n_tok, p.n_seq) * p.n_heads;
    e = gdr::launch_dependent(dla_grad_kernel<DK, DV>, dim3((unsigned)std::min<int64_t>(n, 152)), kGradThreads, GradSmem<DK, DV>::kBytes,
                              stream, wm[0], wm[1], wm[2], wm[3], p, bp, copies, wide(p.dq, p.dk, p.d_k), wide(p.dv, p.dv, p.d_v), n);
    if (e != cudaSuccess) return e;
    if (p.n_heads > p.n_k_heads) {
        const int64_t threads = 2 * p.n_tok * p.n_k_heads * (DK / 8);
        e = gdr::launch_dependent(dla_shared_heads_kernel<DK>, dim3((unsigned)((threads + 255) / 256)), 256, 0, stream, bp.dq, bp.dk, p,
                                  wide(p.dq, p.dk, p.d_k) > 0);
        if (e != cudaSuccess) return e;
    }
    if (p.dg && p.g_stride == 0) return launch_dla_sum_decay(bp.sums, block_slots(p.n_tok, p.n_seq), p.n_heads, p.dg, stream);
    return cudaSuccess;
}

}  // namespace
}  // namespace dla

size_t dla_tc_bwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t n_k_heads, int32_t d_k, int32_t d_v) {
    return dla::layout(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v).bytes;
}

cudaError_t launch_dla_tc_bwd(const DlaArgs &p, cudaStream_t stream) {
    if (p.d_k <= 64) return p.d_v <= 64 ? dla::backward<64, 64>(p, stream) : dla::backward<64, 128>(p, stream);
    return p.d_v <= 64 ? dla::backward<128, 64>(p, stream) : dla::backward<128, 128>(p, stream);
}

cudaError_t read_dla_bwd_flags(unsigned int *flags, bool reset, cudaStream_t stream) {
    return dla::read_flags(flags, reset, stream);
}

}  // namespace kda
