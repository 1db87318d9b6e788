// The walk over a segment that carries the state alone, forward over K and V or in reverse over Q
// and dO (the gradient of the state), on tcgen05. Internal; included by the forward pass (what each
// segment adds to the state) and the backward pass (the state at every block of 128 tokens).
#pragma once

#include <algorithm>
#include <cmath>

#include "kda_dla_tc.h"

namespace kda {
namespace dla {

// one 16 x 16 block of fragments to a swizzled tile, `a` the address of the lane's row
__device__ __forceinline__ void store_matrices(uint32_t a, const uint32_t *f) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(f[0]), "r"(f[1]),
                 "r"(f[2]), "r"(f[3]) : "memory");
}
__device__ __forceinline__ void store_matrices_t(uint32_t a, const uint32_t *f) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(f[0]), "r"(f[1]),
                 "r"(f[2]), "r"(f[3]) : "memory");
}

// How a call is cut into segments
struct Plan {
    int seg;             // tokens of a segment
    int64_t slots;       // of segments
    bool cut;            // some sequence may have more than one
    bool vec_q, vec_k, vec_v, vec_o;  // 16-byte rows
    TileGates *gates;    // [tiles][heads]
    float *states;       // [slots][heads] states at the segments' starts (reverse: gradients at their ends)
    Two *decays;         // [slots][heads] decays over the segments, in two parts
};
// Tiles of a segment, from the call's sizes alone (the sequences' lengths are on the device). Cutting costs
// K and V read once more, what a CTA takes to begin (the time of four tiles) and the join; not cutting
// leaves SMs idle. One sequence: the count of segments whose waves of CTAs take least, in times of a
// tile (64K tokens of 32 heads: 19 segments 636 us, 40 segments 716). Several, of whatever lengths: longer segments cost
// balance, shorter ones beginnings; the sum is least near a square root (20K tokens in two sequences, 8
// heads: 90 us with 12 tiles, 69 with 17, 90 with 30; 60K in four, 32 heads: 569 us with 57 tiles, 524 with
// 69, 606 with 85). Where sequences and heads are two waves by themselves, most sequences stay whole (20K
// tokens in 12 sequences, 32 heads: 198 us with 53 tiles, 166 with 66).
inline int segment_tiles(int64_t n_tok, int32_t n_seq, int32_t n_heads) {
    constexpr int kSMs = 152;
    const int64_t tiles = (n_tok + C - 1) / C;
    if (tiles <= 8) return 8;
    if (n_seq > 1) {
        const double m = std::sqrt(16.0 * (double)tiles * n_heads / kSMs), whole = 2.5 * (double)tiles / n_seq;
        return std::max(8, (int)std::ceil((int64_t)n_seq * n_heads >= 2 * kSMs ? std::max(m, whole) : m));
    }
    struct Last { int64_t tiles; int32_t heads; int best; };
    thread_local Last last{0, 0, 0};
    if (last.tiles == tiles && last.heads == n_heads) return last.best;
    double least = 0;
    int best = 0;
    for (int n = 1; n <= 256 && n * 8 <= tiles + 7; ++n) {
        const int64_t m = (tiles + n - 1) / n, units = (tiles + m - 1) / m * n_heads;
        double cost = (double)((units + kSMs - 1) / kSMs) * (m + 4);
        if (n > 1) cost += (double)((units - n_heads + kSMs - 1) / kSMs) * (0.38 * m + 2.5) + 3;
        if (best == 0 || cost < least) {
            least = cost;
            best = (int)m;
        }
    }
    last = {tiles, n_heads, best};
    return best;
}
// The workspace: the tiles' gates, then, when sequences are cut, the segments' states and decays.
inline size_t gate_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads) {
    return (size_t)n_slots(n_tok, n_seq) * n_heads * sizeof(TileGates);
}
inline size_t plan_bytes(int64_t n_tok, int32_t n_seq, int32_t n_heads, int32_t d_k) {
    const int64_t seg = (int64_t)segment_tiles(n_tok, n_seq, n_heads) * C;
    const size_t units = n_tok > seg ? (size_t)(n_tok / seg + n_seq) * n_heads : 0;
    return (gate_bytes(n_tok, n_seq, n_heads) + units * (state_floats(d_k <= 64 ? 64 : 128) * 4 + sizeof(Two)) + 255) / 256 * 256;
}
inline Plan make_plan(const DlaArgs &p, bool bwd) {
    Plan plan{};
    plan.seg = segment_tiles(p.n_tok, p.n_seq, p.n_heads) * C;
    plan.cut = p.n_tok > plan.seg;
    plan.slots = p.n_tok / plan.seg + p.n_seq;
    plan.vec_q = gdr::rows_vec<__nv_bfloat16>(p.q, p.q_stride, p.in_k);
    plan.vec_k = gdr::rows_vec<__nv_bfloat16>(p.k, p.k_stride, p.in_k);
    plan.vec_v = gdr::rows_vec<__nv_bfloat16>(p.v, p.v_stride, p.in_v);
    plan.vec_o = bwd && gdr::rows_vec<__nv_bfloat16>(p.dout, (int64_t)p.n_heads * p.in_v, p.in_v);
    plan.gates = static_cast<TileGates *>(p.workspace);
    plan.states = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + gate_bytes(p.n_tok, p.n_seq, p.n_heads));
    plan.decays = reinterpret_cast<Two *>(plan.states + (size_t)plan.slots * p.n_heads * state_floats(p.d_k <= 64 ? 64 : 128));
    return plan;
}

// Heads of a number of channels that is no multiple of eight lie where no tensor copy can fetch them, and by
// threads a tile takes 10000 cycles to arrive. Such inputs are copied once, to rows of 8 ceil(d / 8) channels, behind the
// rest of the workspace (20K tokens of 4 / 32 heads, d_k 33, d_v 64: 1376 us by threads, 148 with the copy).
constexpr int padded(int d) { return (d + 7) / 8 * 8; }
inline size_t aligned_bytes(int64_t n_tok, int heads, int d) { return d % 8 ? ((size_t)n_tok * heads * padded(d) * 2 + 255) / 256 * 256 : 0; }
inline size_t copies_bytes(int64_t n_tok, int32_t n_heads, int32_t n_k_heads, int32_t d_k, int32_t d_v, bool bwd) {
    return 2 * aligned_bytes(n_tok, n_k_heads, d_k) + (bwd ? 2 : 1) * aligned_bytes(n_tok, n_heads, d_v);
}
struct Rows { const __nv_bfloat16 *from; int64_t stride; uint4 *to; int heads, d; };
struct RowCopies { Rows r[4]; };
static __global__ void __launch_bounds__(256) dla_align_kernel(const RowCopies all, int64_t n_tok) {
    const Rows &r = all.r[blockIdx.y];
    const int per = padded(r.d) / 8;  // eight channels a thread
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / per;
    if (row >= n_tok * r.heads) return;
    const int c = (int)(i % per) * 8;
    const uint16_t *from = reinterpret_cast<const uint16_t *>(r.from) + row / r.heads * r.stride + row % r.heads * r.d + c;
    uint32_t x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = c + e < r.d ? from[e] : 0;
    r.to[i] = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
}
// `at`: copies_bytes of the workspace
inline cudaError_t align_inputs(DlaArgs &p, char *at, bool bwd, cudaStream_t stream) {
    RowCopies all{};
    int n = 0;
    int64_t most = 0;
    auto take = [&](const void *&x, int64_t stride, int heads, int d) {
        Rows &r = all.r[n++];
        r = {static_cast<const __nv_bfloat16 *>(x), stride, reinterpret_cast<uint4 *>(at), heads, d};
        x = at;
        at += aligned_bytes(p.n_tok, heads, d);
        most = std::max(most, p.n_tok * heads * (padded(d) / 8));
    };
    if (p.d_k % 8) {
        take(p.q, p.q_stride, p.n_k_heads, p.d_k);
        take(p.k, p.k_stride, p.n_k_heads, p.d_k);
        p.in_k = padded(p.d_k);
        p.q_stride = p.k_stride = (int64_t)p.n_k_heads * p.in_k;
    }
    if (p.d_v % 8) {
        take(p.v, p.v_stride, p.n_heads, p.d_v);
        if (bwd) take(p.dout, (int64_t)p.n_heads * p.d_v, p.n_heads, p.d_v);
        p.in_v = padded(p.d_v);
        p.v_stride = (int64_t)p.n_heads * p.in_v;
    }
    if (n == 0) return cudaSuccess;
    dla_align_kernel<<<dim3((unsigned)((most + 255) / 256), n), 256, 0, stream>>>(all, p.n_tok);
    count_launches(1);
    return cudaGetLastError();
}

// The gates of every tile and head: a warp four heads of a tile, whose decays are neighbours in memory and
// whose scans run beside each other (64K tokens of 32 heads: 31 us with a head a warp, 14 with four; 17 since a
// tile's decay is formed in two parts).
static __global__ void __launch_bounds__(256) dla_gates_kernel(const DlaArgs p, TileGates *out) {
    gdr::let_next_kernel_start();
    const int quads = (p.n_heads + 3) / 4;
    const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), slot = unit / quads;
    if (slot >= n_slots(p.n_tok, p.n_seq)) return;
    const Chunk ch = find_chunk(p.cu_seqlens, p.n_seq, slot);
    if (ch.len == 0) return;
    const int r = 2 * (threadIdx.x & 31), h0 = (int)(unit % quads) * 4, n = min(4, p.n_heads - h0);
    float2 x[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float *g = p.g + (ch.t0 + r) * p.g_stride + h0 + h;
        x[h] = make_float2(h < n && r < ch.len ? g[0] : 0.f, h < n && r + 1 < ch.len ? g[p.g_stride] : 0.f);
    }
    TileGates *to = out + slot * p.n_heads + h0;
#pragma unroll
    for (int h = 0; h < 4; ++h)
        if (h < n) form_gates(x[h], p.scale, to + h);
}
inline cudaError_t launch_gates(const DlaArgs &p, const Plan &plan, cudaStream_t stream) {
    const int64_t units = n_slots(p.n_tok, p.n_seq) * ((p.n_heads + 3) / 4);
    dla_gates_kernel<<<(unsigned)((units + 7) / 8), 256, 0, stream>>>(p, plan.gates);
    count_launches(1);
    return cudaGetLastError();
}

// NC key channels from c0 on of one value channel: a state of the workspace
template <int NC>
__device__ __forceinline__ void load_state(float *st, const float *from, int dv, int c0) {
#pragma unroll
    for (int i = 0; i < NC; i += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(from + (c0 + i) / 4 * 512 + dv * 4);
        st[i] = x.x; st[i + 1] = x.y; st[i + 2] = x.z; st[i + 3] = x.w;
    }
}
template <int NC>
__device__ __forceinline__ void store_state(const float *st, float *to, int dv, int c0) {
#pragma unroll
    for (int i = 0; i < NC; i += 4)
        *reinterpret_cast<float4 *>(to + (c0 + i) / 4 * 512 + dv * 4) = make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
}
// the caller's [d_k][d_v] (NULL: zeros)
template <int NC>
__device__ __forceinline__ void load_given(float *st, const float *from, int d_k, int d_v, int dv, int c0) {
    const int n = from && dv < d_v ? d_k - c0 : 0;
    const float *x = from + (int64_t)c0 * d_v + dv;
#pragma unroll
    for (int i = 0; i < NC; ++i, x += d_v) st[i] = i < n ? *x : 0.f;
}
template <int NC>
__device__ __forceinline__ void store_given(const float *st, float *to, int d_k, int d_v, int dv, int c0) {
    const int n = dv < d_v ? d_k - c0 : 0;
    float *x = to + (int64_t)c0 * d_v + dv;
#pragma unroll
    for (int i = 0; i < NC; ++i, x += d_v)
        if (i < n) *x = st[i];
}

// warps: 0 issues products, 1 loads, 4..11 scale the values (every other tile each four), 12..19 read the sums
constexpr int kSegmentThreads = 640;
constexpr int kSum = 2;  // tiles that are summed in tensor memory

template <int DK>
struct SegmentSmem {
    static constexpr int kKey = DK / 64 * kHalf, kVal = 2 * kHalf;
    static constexpr int K = 0, V = kKey, Gate = V + kVal, kStage = Gate + 2048;
    static constexpr int kStages = 6, Bars = kStages * kStage;
    static constexpr int Full = 0, Empty = kStages, VpFull = 2 * kStages, VpEmpty = VpFull + 2, DsFull = VpEmpty + 2,
                         DsEmpty = DsFull + 2, Drain = DsEmpty + 2, Partial = Drain + 1, kBars = Partial + 1;
    static constexpr int kBytes = Bars + 8 * kBars + 16 + 1024;  // the base is rounded up to 1024
    static_assert(sizeof(TileGates) <= 2048 && kBytes <= 227 * 1024, "fits an SM");
};

// What a segment adds to the state, from a state of zero, and its decay. The values' factors reach to the
// segment's end, so that the sum over tiles stays in tensor memory, from the last tile to the first (REV,
// the gradient: from the first to the last); every second tile it is added to registers, because the
// tensor cores drop bits below a running sum's last place, and the smallest planes' products come first for
// the same reason. Three planes of the values times their factors, where the forward pass's last walk has room
// for two: a state is read by every later token and dg is summed from it (8192 tokens: dg off by
// 5.5e-6 of its norm with two, 3.1e-6 with three, dh0 by 4.7e-6 and 0.3e-6; the walk takes 164 us and
// 172 us). The last segment of the walk hands on to
// none and is left out.
template <int DK, bool REV>
__device__ __forceinline__ void segment_walk(const CUtensorMap &tm_key, const CUtensorMap &tm_val, const DlaArgs &p,
                                             const Plan &plan, bool copies, unsigned unit) {
    using L = SegmentSmem<DK>;
    constexpr int S = L::kStages;
    extern __shared__ __align__(1024) char smem_raw[];
    char *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_u32(smem);
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };  // equal over a warp, and told so
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int head = unit % p.n_heads, kh = head / (p.n_heads / p.n_k_heads);
    const int64_t slot = unit / p.n_heads;
    const Segment sg = find_segment(p.cu_seqlens, p.n_seq, slot, plan.seg);
    if (sg.len == 0 || (REV ? sg.index == 0 : sg.last)) {
        gdr::wait_for_previous_kernel();  // whoever waits for this kernel waits for that one
        return;
    }
    const int nc = uniform((int)((sg.len + C - 1) / C));
    auto bar = [&](int i) { return base + L::Bars + 8 * i; };
    auto tile = [&](int n) { return REV ? n : nc - 1 - n; };  // the n-th of the walk
    auto rows_of = [&](int c) { return (int)min((int64_t)C, sg.len - (int64_t)c * C); };
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            ptx::mbar_init(bar(L::Full + i), 1);
            ptx::mbar_init(bar(L::Empty + i), 1 + 8);  // all eight scaling warps read the decay
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(L::VpFull + i), 4);
            ptx::mbar_init(bar(L::VpEmpty + i), 1);
            ptx::mbar_init(bar(L::DsFull + i), 1);
            ptx::mbar_init(bar(L::DsEmpty + i), 8);
        }
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
    if (warp == 0) {
        constexpr uint32_t id = ptx::idesc_bf16(128, DK, 0, 1);
        const uint32_t leader = ptx::elect_one();
        const uint64_t k0 = ptx::sdesc_sw128(base + L::K, kHalf, 1024);
        int s = 0;
#pragma unroll 1
        for (int n = 0; n < nc; ++n) {
            const int b = (n / kSum) & 1;  // the buffer of this sum
            wait(L::VpFull + (n & 1), n >> 1);
            if (n % kSum == 0 && n >= 2 * kSum) wait(L::DsEmpty + b, n / (2 * kSum) - 1);
            ptx::tc_fence_after();
            const uint32_t at = (uint32_t)s * (L::kStage / 16), more = n % kSum != 0;
            if (leader) {
#pragma unroll
                for (int i = 2; i >= 0; --i)
#pragma unroll
                    for (int k = 0; k < C / 16; ++k)
                        ptx::umma_ts(tmem + b * 128, tmem + 256 + (n & 1) * 96 + i * 32 + 8 * k, k0 + (at + 128 * k), id,
                                     i < 2 || k > 0 ? 1 : more);
                if ((n + 1) % kSum == 0 || n + 1 == nc) ptx::umma_commit(bar(L::DsFull + b));
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
        for (int n = 0; n < nc; ++n) {
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
    } else if (warp >= 4 && warp < 12) {
        // the exponent of the decay from the tile's end to the walk's, in fixed point; past -2048 it may be any
        int64_t past = 0;
        float bad = 0.f;
        const int turn = (warp - 4) >> 2;
        for (int n = 0; n < nc; ++n) {
            const int s = n % S;
            wait(L::Full + s, n / S);
            const TileGates *g = reinterpret_cast<const TileGates *>(smem + s * L::kStage + L::Gate);
            if ((n & 1) == turn) {
                auto ready = [&] {
                    if (n >= 2) wait(L::VpEmpty + turn, (n >> 1) - 1);
                    ptx::tc_fence_after();
                };
                if (32 * (warp & 3) < p.d_v)  // other lanes' rows are not read
                    scale_values<3>(base + s * L::kStage + L::V, tmem, 256 + turn * 96, REV ? g->gam : g->del, exp2_fixed(past) + bad, ready);
                else ready();
                ptx::tc_fence_before();
                warp_arrive(bar(L::VpFull + turn));
            }
            past = max(past + g->sum, -((int64_t)2048 << kPoint));
            bad += nan_of(*g);
            warp_arrive(bar(L::Empty + s));
        }
        if (tid == 128) {
            const Two beyond = exp2_fixed_parts(past);
            plan.decays[(size_t)slot * p.n_heads + head] = {beyond.hi + bad, beyond.lo};
        }
    } else if (warp >= 12) {
        constexpr int NC = DK / 2;  // key channels of a thread
        const int dv = (warp & 3) * 32 + lane, part = (warp - 12) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        float st[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) st[i] = 0.f;
        for (int n = 0; n * kSum < nc; ++n) {
            wait(L::DsFull + (n & 1), n >> 1);
            ptx::tc_fence_after();
            if (32 * (warp & 3) < p.d_v)
#pragma unroll
                for (int i = 0; i < NC; i += 16) {
                    float d[16];
                    ptx::tmem_ld16(lanes + (n & 1) * 128 + part * NC + i, reinterpret_cast<uint32_t *>(d));
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) st[i + j] += d[j];
                }
            ptx::tc_fence_before();
            warp_arrive(bar(L::DsEmpty + (n & 1)));
        }
        store_state<NC>(st, plan.states + ((size_t)slot * p.n_heads + head) * state_floats(DK), dv, part * NC);
    }
    __syncwarp();
    __syncthreads();
    if (warp == 0) ptx::tmem_dealloc(tmem, 512);
}

// The plan as one direction's walk sees it: the reverse one's states and decays lie behind the forward one's.
template <int DK>
__host__ __device__ __forceinline__ Plan of_walk(Plan plan, const DlaArgs &p, bool rev) {
    const size_t units = (size_t)plan.slots * p.n_heads;
    if (rev) {
        plan.states += units * state_floats(DK);
        plan.decays += units;
    }
    return plan;
}

// Forward, or with twice the blocks in reverse first and forward
template <int DK>
__global__ void __launch_bounds__(kSegmentThreads, 1)
    dla_segments_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const DlaArgs p,
                        const Plan plan, bool copies) {
    gdr::let_next_kernel_start();
    const unsigned n = (unsigned)plan.slots * p.n_heads, rest = gridDim.x - n;
    if (blockIdx.x < rest) segment_walk<DK, true>(tm_q, tm_o, p, of_walk<DK>(plan, p, true), copies, blockIdx.x);
    else segment_walk<DK, false>(tm_k, tm_v, p, plan, copies, blockIdx.x - rest);
}

// The states at the segments' starts (reverse: the gradients at their ends), in place of what the
// segments add: 16 bytes of a sequence's and head's state a thread, segment after segment.
template <int DK>
__global__ void __launch_bounds__(256) dla_join_kernel(const DlaArgs p, const Plan both) {
    gdr::let_next_kernel_start();
    const bool rev = blockIdx.y == 1;
    const Plan plan = of_walk<DK>(both, p, rev);
    constexpr int kBlocks = state_floats(DK) / 4 / 256;
    const int i = (blockIdx.x % kBlocks) * 256 + threadIdx.x;
    const int head = blockIdx.x / kBlocks % p.n_heads, seq = blockIdx.x / kBlocks / p.n_heads;
    const int64_t len = p.cu_seqlens[seq + 1] - p.cu_seqlens[seq], m = (len + plan.seg - 1) / plan.seg;
    if (m < 2) {
        gdr::wait_for_previous_kernel();  // whoever waits for this kernel waits for that one
        return;
    }
    const int dv = i & 127, c = i >> 7 << 2;
    const float *given = rev ? p.dh_final : p.h0;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (given && dv < p.d_v) {
        const float *from = given + ((int64_t)seq * p.n_heads + head) * p.d_k * p.d_v + dv;
        if (c < p.d_k) x.x = from[(int64_t)c * p.d_v];
        if (c + 1 < p.d_k) x.y = from[(int64_t)(c + 1) * p.d_v];
        if (c + 2 < p.d_k) x.z = from[(int64_t)(c + 2) * p.d_v];
        if (c + 3 < p.d_k) x.w = from[(int64_t)(c + 3) * p.d_v];
    }
    const int64_t slot0 = segment_base(p.cu_seqlens, seq, plan.seg);
    gdr::wait_for_previous_kernel();
    auto unit = [&](int64_t n) { return (size_t)(slot0 + (rev ? m - 1 - n : n)) * p.n_heads + head; };
    auto at = [&](int64_t n) { return reinterpret_cast<float4 *>(plan.states + unit(n) * state_floats(DK)) + i; };
    Factors decays;
    for (int64_t n0 = 0; n0 < m; n0 += 4) {
        float4 add[4];
        Two decay[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n0 + j + 1 < m) {  // the last one hands on to none
                add[j] = *at(n0 + j);
                decay[j] = plan.decays[unit(n0 + j)];
            }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n0 + j >= m) break;
            *at(n0 + j) = x;
            if (n0 + j + 1 == m) break;
            const float w = decays.next(decay[j]);
            x.x = fmaf(w, x.x, add[j].x);
            x.y = fmaf(w, x.y, add[j].y);
            x.z = fmaf(w, x.z, add[j].z);
            x.w = fmaf(w, x.w, add[j].w);
        }
    }
}

template <int DK>
cudaError_t launch_segments(const DlaArgs &p, const Plan &plan, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                            const CUtensorMap &o, bool copies, int walks, cudaStream_t stream) {
    const cudaError_t e = gdr::launch_dependent(dla_segments_kernel<DK>, dim3((unsigned)(walks * plan.slots * p.n_heads)), kSegmentThreads,
                                                SegmentSmem<DK>::kBytes, stream, q, k, v, o, p, plan, copies);
    if (e != cudaSuccess) return e;
    return gdr::launch_dependent(dla_join_kernel<DK>, dim3((unsigned)(state_floats(DK) / 1024 * p.n_heads * p.n_seq), walks), 256, 0,
                                 stream, p, plan);
}

}  // namespace dla
}  // namespace kda
