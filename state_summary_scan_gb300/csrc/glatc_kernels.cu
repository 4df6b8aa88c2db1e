// glatc_kernels.cu -- linear attention with a decay for each head and a carried state in chunks of 64 tokens on
// the tensor cores (tcgen05 + TMA): ragged prompts in bf16, Dk in {64, 128}, any Dv.
//
// With b_t the running sum of a chunk's gates (b_63 its end) and S the state before the chunk:
//     O  = scale (e^b o (Q S) + P V),   P[t][s] = (q_t.k_s) e^{b_t - b_s} for s <= t
//     S' = e^{b_63} S + K^T V~,         V~_t = e^{b_63 - b_t} v_t
// gla_walk_kernel: one CTA per (sequence, head, 128 columns of values) walks the sequence's chunks.  Everything
// is transposed, a value column a lane: V~^T and S^T enter as A operands from tensor memory, into which the lanes
// write them, and O^T, K^T V~ leave as rows of it.  The state itself stays in registers in fp32: K^T V~ is formed
// for each chunk by itself, so that no product waits for the state but Q S, and the state's sum is rounded to
// nearest, with no run of accumulations.  The decays within a chunk are at most 1 wherever the gates are at most 0: they are formed
// from differences of running sums in fixed point, within 32 tokens directly, and across them through the border.
//
// Where the sequences and heads are too few to fill the GPU, long sequences are cut into segments.  A segment's
// map of the state is S -> e^{sum g} S + dS: a first launch walks the first segment, and the inner ones from zero
// without outputs; a second one walks the segments after the first, each from the state that it folds together
// from the first one's end and the maps between.
//
// Rounding: K, Q and V enter as they are; V~ as the sum of two bf16, or of three (all 24 bits) where the pool is
// fp32, because its errors reach the state undamped.  S and P are rounded once to bf16: they only enter O,
// which is rounded to bf16 anyway.
#include <cstdio>

#include "gla.cuh"
#include "tc_walk.cuh"

namespace rmcp {
namespace gla {

using namespace tc;
using gds::T8;
using gds::by_length;
using gds::map_of;
using gds::mma_ts;
using gds::tmem_ld;
using gds::tmem_st;
using gds::wait;
using gds::warp_arrive;
using gds::zero_rows;

namespace {

constexpr float kForget = 110.f;             // e^-110 is 0 in fp32: lower gates are raised to -110
constexpr float kFixed = 1099511627776.f;    // gates in units of 2^-40
constexpr int kSub = 32;                     // tokens whose decays are formed pair by pair
constexpr int kMostSegments = 16;
constexpr int kMostStates = 320;             // of segments: see tc_workspace_bytes()

// A chunk's gates in shared memory, in floats
constexpr int kOut = 0;      // scale e^{b_t}
constexpr int kDec = 64;     // e^{b_63 - b_t}
constexpr int kLocal = 128;  // b_t from the start of its 32 tokens
constexpr int kCross = 192;  // e^{b_31 - b_s} of the first 32
constexpr int kEnd = 224;    // the state's decay: S + kEnd S (kNear), or kEnd S
constexpr int kNear = 225;
constexpr uint32_t kGateBytes = 1024;
constexpr int kGateRing = 8;
constexpr int kStages = 3;
constexpr int kGroups = 4;                                  // groups of four warps of the state
constexpr int kWalkThreads = (4 * kGroups + 4 + 2 + 2) * 32;  // and four output warps, two of scores, the products', the copies' and gates'
constexpr int kOutWarp = 4 * kGroups, kScoreWarp = kOutWarp + 4, kMmaWarp = kScoreWarp + 2;

template <int DK>
struct WalkSmem {
    static constexpr int NP = DK / 64;
    // a stage: for each 64 dimensions 64 rows of Q, then 64 of K (one operand of 128 rows); then V
    static constexpr uint32_t panel = 2 * T8, V = NP * panel, stage = V + 2 * T8;
    static constexpr uint32_t P = kStages * stage, OUT = P + T8, GATES = OUT + 2 * T8;
    static constexpr size_t bytes = GATES + kGateRing * kGateBytes + 1024;
};
static_assert(WalkSmem<128>::bytes <= 227 * 1024, "shared memory of a CTA");

// Tensor-memory columns: K^T V~ transposed, scores, Q S and P V transposed (fp32), then S^T and V~^T (bf16 pairs)
constexpr uint32_t TM_D = 0, TM_SC = 128, TM_O1 = 192, TM_O2 = 256, TM_S = 320, TM_V = 384;

struct WalkBars {
    uint64_t full[kStages], empty[kStages], gates[kGateRing];
    uint64_t scores, scores_free, p_ready, ready, d_done, o_done, o_free, fixed;
};

enum class Part { whole, first, rest };  // as the delta rule's walk divides the sequences (gdstc_kernels.cu)
struct Segments {
    int chunks;    // of a segment
    int most;      // segments of the longest sequence
    float* ends;   // [S][H][most][Dk][Dv]: dS of the inner segments, the first one's end
    float* fades;  // [S][H][most]: e^{sum g}
};
__device__ __forceinline__ int64_t segment_at(const Args& a, const Segments& g, int seq, int h, int j) {
    return (int64_t(seq) * a.H + h) * g.most + j;
}

// The loads before a tmem_wait_ld() have arrived: nothing that uses them moves above it.
template <int N>
__device__ __forceinline__ void arrived(uint32_t* r) {
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

template <int DK, typename TS, Part kPart>
__global__ void __launch_bounds__(kWalkThreads, 1)
    gla_walk_kernel(const __grid_constant__ Args a, const Segments seg, const __grid_constant__ CUtensorMap mq,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
    constexpr int NP = DK / 64;
    constexpr int GC = DK / kGroups;      // state rows of a group
    constexpr int GT = kChunk / kGroups;  // tokens of a group
    constexpr int kParts = sizeof(TS) == 4 ? 3 : 2;  // of V~
    using L = WalkSmem<DK>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    __shared__ __align__(8) WalkBars bar;
    __shared__ uint32_t tmem_slot;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blocks = (a.Dv + 127) / 128;
    const int h = blockIdx.x / blocks, v0 = blockIdx.x % blocks * 128, nv = min(a.Dv - v0, 128);
    const int si = kPart == Part::whole ? by_length(a, blockIdx.y) : int(blockIdx.y);
    const Seq sq = sequence(a, si);
    const int all = (sq.len + kChunk - 1) / kChunk;  // the sequence's chunks
    const int j = kPart == Part::whole ? 0 : int(blockIdx.z) + (kPart == Part::rest ? 1 : 0);
    const int c_first = kPart == Part::whole ? 0 : j * seg.chunks;
    // the sequence's last segment (the last one that there is takes what a sequence has beyond max_len)
    const bool ends = kPart == Part::whole || j == seg.most - 1 || c_first + seg.chunks >= all;
    const int chunks = (ends ? all : c_first + seg.chunks) - c_first;
    if (kPart != Part::whole && j > 0 && (sq.slot < 0 || chunks <= 0)) return;
    if (kPart == Part::first && j > 0 && ends) return;
    const bool outs = kPart != Part::first || j == 0;  // it has outputs
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + ((int64_t(sq.begin) + int64_t(c_first) * kChunk) * a.H + h) * a.Dv + v0;
    const int64_t os = int64_t(a.H) * a.Dv;
    TS* st = static_cast<TS*>(a.state) + (int64_t(max(sq.slot, 0)) * a.H + h) * DK * a.Dv + v0;
    if (kPart != Part::rest && j == 0)
        zero_others(a, si, sq, static_cast<__nv_bfloat16*>(a.o) + int64_t(h) * a.Dv + v0, nv, tid, kWalkThreads);
    if (sq.slot < 0) {  // padding
        zero_outputs(o, os, sq.len, nv, tid, kWalkThreads);
        return;
    }
    if (sq.len == 0) {
        if (sq.fresh)
            for (int i = tid; i < DK * nv; i += kWalkThreads) st[int64_t(i / nv) * a.Dv + i % nv] = from_f32<TS>(0.f);
        return;
    }
    const int last = sq.len - (all - 1) * kChunk;  // tokens of the sequence's last chunk
    const bool ragged = ends && last < kChunk;
    const int quads = (nv + 31) / 32;  // quadrants of tensor-memory lanes with columns

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&bar.full[i]), 1);
            mbar_init(smem_u32(&bar.empty[i]), 1 + quads * kGroups);
        }
        for (int i = 0; i < kGateRing; ++i) mbar_init(smem_u32(&bar.gates[i]), 1);
        mbar_init(smem_u32(&bar.scores), 1);
        mbar_init(smem_u32(&bar.scores_free), 2);
        mbar_init(smem_u32(&bar.p_ready), 2);
        mbar_init(smem_u32(&bar.ready), quads * kGroups);
        mbar_init(smem_u32(&bar.d_done), 1);
        mbar_init(smem_u32(&bar.o_done), 1);
        mbar_init(smem_u32(&bar.o_free), quads);
        mbar_init(smem_u32(&bar.fixed), quads * kGroups);
        mbar_fence_init();
    }
    if (warp == 0) tmem_alloc(smem_u32(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    bool dead = false;
    auto gates_of = [&](int c) {  // the chunk's gates, once they are there
        wait(&bar.gates[c % kGateRing], (c / kGateRing) & 1, dead);
        return reinterpret_cast<const float*>(smem + L::GATES + (c % kGateRing) * kGateBytes);
    };
    auto wait_full = [&](int c) { wait(&bar.full[c % kStages], (c / kStages) & 1, dead); };

    if (warp < kOutWarp) {
        // ---- the state: a lane is a value column, a group has a quarter of its rows, and of a chunk's tokens
        if ((warp & 3) < quads) {
            const int grp = warp >> 2, row = 32 * (warp & 3) + lane;
            const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);
            const bool live = row < nv;
            const int r0 = grp * GC;
            uint64_t S[GC / 2];  // pairs of rows
            {
                auto rows = [&](auto at) {
#pragma unroll
                    for (int i = 0; i < GC / 2; ++i) S[i] = live ? pair(at(r0 + 2 * i), at(r0 + 2 * i + 1)) : 0;
                };
                if (kPart == Part::whole || (kPart == Part::first && j == 0)) {
                    if (sq.fresh) rows([](int) { return 0.f; });
                    else rows([&](int r) { return to_f32(st[int64_t(r) * a.Dv + row]); });
                } else if (kPart == Part::first) {
                    rows([](int) { return 0.f; });
                } else {  // the first segment's end, through the maps of those up to this one
                    const float* e = seg.ends + segment_at(a, seg, si, h, 0) * DK * a.Dv + v0 + row;
                    rows([&](int r) { return e[int64_t(r) * a.Dv]; });
                    for (int i = 1; i < j; ++i) {
                        const float f = seg.fades[segment_at(a, seg, si, h, i)];
                        e += int64_t(DK) * a.Dv;
                        if (live) {
#pragma unroll
                            for (int u = 0; u < GC / 2; ++u)
                                S[u] = fma2(pair(f, f), S[u], pair(e[int64_t(r0 + 2 * u) * a.Dv], e[int64_t(r0 + 2 * u + 1) * a.Dv]));
                        }
                    }
                }
            }
            // S <- e^{b_63} S + K^T V~ of chunk c
            auto update = [&](int c) {
                const float* gates = gates_of(c);
                const uint64_t end = pair(gates[kEnd], gates[kEnd]);
                const bool near = gates[kNear] != 0.f;
                uint32_t d[GC];
                tmem_ld<GC>(tl + TM_D + r0, d);
                arrived<GC>(d);
                if (near) {  // near 1 the decay's distance from 1 is what is known to all its bits
#pragma unroll
                    for (int i = 0; i < GC / 2; ++i) S[i] = add2(fma2(end, S[i], pair(d[2 * i], d[2 * i + 1])), S[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < GC / 2; ++i) S[i] = fma2(end, S[i], pair(d[2 * i], d[2 * i + 1]));
                }
            };
            for (int c = 0; c < chunks; ++c) {
                const uint8_t* stage = smem + (c % kStages) * L::stage;
                const float* gates = gates_of(c);
                wait_full(c);
                const bool tail = ragged && c == chunks - 1;
                const int n = tail ? last : kChunk;
                if (tail) {  // keys and values past the sequence's end are other tokens': they must not meet a zero as NaN
                    const int at = (grp * quads + (warp & 3)) * 32 + lane, threads = 32 * quads * kGroups;
                    for (int p = 0; p < NP; ++p) zero_rows(smem + (c % kStages) * L::stage + p * L::panel + T8, 1, n, at, threads);
                    zero_rows(smem + (c % kStages) * L::stage + L::V, 2, n, at, threads);
                    fence_async_smem();
                    warp_arrive(&bar.fixed, lane);
                }
                uint32_t v[kParts][GT / 2];
#pragma unroll
                for (int i = 0; i < GT / 2; ++i) {
                    const int t = GT * grp + 2 * i;
                    const uint32_t x = *reinterpret_cast<const uint16_t*>(stage + L::V + sw_off(64, t, row)),
                                   y = *reinterpret_cast<const uint16_t*>(stage + L::V + sw_off(64, t + 1, row));
                    uint64_t w = mul2(pair(x << 16, y << 16), *reinterpret_cast<const uint64_t*>(gates + kDec + t));
                    if (tail) {
                        uint32_t w0, w1;
                        unpair(w, w0, w1);
                        w = pair(t < n ? w0 : 0u, t + 1 < n ? w1 : 0u);
                    }
                    if (kParts == 3) split2(w, v[0][i], v[1][i], v[kParts - 1][i]);
                    else split2(w, v[0][i], v[1][i]);
                }
                warp_arrive(&bar.empty[c % kStages], lane);
                if (c > 0) {
                    wait(&bar.d_done, (c - 1) & 1, dead);
                    tc_fence_after();
                }
#pragma unroll
                for (int p = 0; p < kParts; ++p) tmem_st<GT / 2>(tl + TM_V + 32 * p + GT / 2 * grp, v[p]);
                if (c > 0) update(c - 1);
                if (outs) {
                    uint32_t s[GC / 2];
#pragma unroll
                    for (int i = 0; i < GC / 2; ++i) s[i] = pack2(S[i]);
                    tmem_st<GC / 2>(tl + TM_S + r0 / 2, s);
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&bar.ready, lane);
            }
            wait(&bar.d_done, (chunks - 1) & 1, dead);
            tc_fence_after();
            update(chunks - 1);
            tc_fence_before();
            if (live && (ends || kPart == Part::first)) {
                float* to = ends ? nullptr : seg.ends + segment_at(a, seg, si, h, j) * DK * a.Dv + v0 + row;
#pragma unroll
                for (int i = 0; i < GC / 2; ++i) {
                    uint32_t x[2];
                    unpair(S[i], x[0], x[1]);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int64_t at = int64_t(r0 + 2 * i + u) * a.Dv;
                        if (ends) st[at + row] = from_f32<TS>(__uint_as_float(x[u]));
                        else to[at] = __uint_as_float(x[u]);
                    }
                }
            }
        }
    } else if (warp < kScoreWarp) {
        // ---- the outputs: a lane is a value column; whole chunks leave as tiles, the last one by rows
        const int w = warp & 3, row = 32 * w + lane;
        if (outs && w < quads) {
            const uint32_t tl = tmem + (uint32_t(32 * w) << 16);
            uint8_t* tile = smem + L::OUT;
            for (int c = 0; c < chunks; ++c) {
                const float* gates = gates_of(c);
                wait(&bar.o_done, c & 1, dead);
                tc_fence_after();
                uint32_t y[kChunk / 2];
#pragma unroll
                for (int t0 = 0; t0 < kChunk; t0 += 16) {
                    uint32_t p[32];
                    tmem_ld<16>(tl + TM_O1 + t0, p);
                    tmem_ld<16>(tl + TM_O2 + t0, p + 16);
                    arrived<32>(p);
#pragma unroll
                    for (int i = 0; i < 16; i += 2)
                        y[(t0 + i) / 2] = pack2(fma2(*reinterpret_cast<const uint64_t*>(gates + kOut + t0 + i), pair(p[i], p[i + 1]), pair(p[16 + i], p[17 + i])));
                }
                tc_fence_before();
                warp_arrive(&bar.o_free, lane);  // the accumulators and the gates have been read
                // the store of the chunk before has read the staging
                if (warp == kOutWarp && lane == 0) bulk_wait_read();
                asm volatile("bar.sync 1, %0;" ::"r"(32 * quads) : "memory");
#pragma unroll
                for (int i = 0; i < kChunk; ++i)
                    *reinterpret_cast<uint16_t*>(tile + (row >> 6) * T8 + sw_off(64, i, row & 63)) =
                        uint16_t(i & 1 ? y[i / 2] >> 16 : y[i / 2] & 0xffffu);
                const bool whole = c < chunks - 1 || !ragged;
                if (whole) fence_async_smem();
                asm volatile("bar.sync 1, %0;" ::"r"(32 * quads) : "memory");
                if (whole) {
                    if (warp == kOutWarp && lane == 0) {
                        for (int p = 0; p < (nv + 63) / 64; ++p)
                            tma_store_3d(&mo, smem_u32(tile + p * T8), v0 + 64 * p, h, sq.begin + (c_first + c) * kChunk);
                        bulk_commit();
                    }
                } else {
                    for (int i = w * 32 + lane; i < last * 16; i += 32 * quads) {
                        const int t = i >> 4, e = (i & 15) * 8;
                        if (e < nv)
                            *reinterpret_cast<uint4*>(o + (int64_t(c) * kChunk + t) * os + e) =
                                *reinterpret_cast<const uint4*>(tile + sw_chunk(64, t, e >> 3));
                    }
                }
            }
            if (warp == kOutWarp && lane == 0) bulk_wait_read();  // shared memory is read before the CTA ends
        }
    } else if (warp < kMmaWarp) {
        // ---- the scores: a lane is a token's row
        if (outs) {
            const int half = warp & 3, t = 32 * half + lane;  // (kScoreWarp is a multiple of four)
            const uint32_t tl = tmem + (uint32_t(32 * half) << 16) + TM_SC;
            for (int c = 0; c < chunks; ++c) {
                const float* gates = gates_of(c);
                wait(&bar.scores, c & 1, dead);
                tc_fence_after();
                const float bt = gates[kLocal + t];
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    uint32_t y[16];
                    if (part > half) {  // the first tokens do not see the second ones
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = 0;
                    } else {
                        uint32_t x[32];
                        tmem_ld<32>(tl + 32 * part, x);
                        arrived<32>(x);
                        if (part < half) {
                            const float f = a.scale * __expf(bt);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                y[i] = pack2(mul2(mul2(pair(f, f), pair(x[2 * i], x[2 * i + 1])), *reinterpret_cast<const uint64_t*>(gates + kCross + 2 * i)));
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float m[2];
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const int s = 2 * i + u;
                                    m[u] = s <= lane ? a.scale * __uint_as_float(x[s]) * __expf(bt - gates[kLocal + 32 * part + s]) : 0.f;
                                }
                                y[i] = pack2(m[0], m[1]);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4*>(smem + L::P + sw_chunk(64, t, 4 * part + i)) = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                }
                tc_fence_before();
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&bar.scores_free));
                    mbar_arrive(smem_u32(&bar.p_ready));
                }
            }
        }
    } else if (warp == kMmaWarp) {
        // ---- the products, in order: Q K^T a chunk ahead, Q S, P V, K^T V~.  The whole warp walks the loop and one
        // elected lane issues.
        const uint32_t base = smem_u32(smem);
        constexpr uint32_t kSc = idesc_bf16(128, 64, 0, 0), kTS = idesc_bf16(128, 64, 0, 0), kPV = idesc_bf16(128, 64, 1, 0),
                           kTD = idesc_bf16(128, DK, 0, 1);
        auto scores = [&](int c) {  // rows 0 .. 63: Q K^T (64 .. 127: K K^T, not read)
            const uint32_t at = base + (c % kStages) * L::stage;
            const uint64_t d = sdesc(at, 16, 1024), dk = sdesc(at + T8, 16, 1024);
            wait_full(c);
            if (c > 0) wait(&bar.scores_free, (c - 1) & 1, dead);
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {
                    const uint32_t off = (k >> 2) * L::panel + (k & 3) * 32;
                    mma_bf16(tmem + TM_SC, desc_plus(d, off), desc_plus(dk, off), kSc, k > 0);
                }
                mma_commit(smem_u32(&bar.scores));
            }
            __syncwarp();
        };
        if (outs) scores(0);
        for (int c = 0; c < chunks; ++c) {
            const uint32_t at = base + (c % kStages) * L::stage;
            const uint64_t dq = sdesc(at, 16, 1024), dk = sdesc(at + T8, L::panel, 1024), dv = sdesc(at + L::V, T8, 1024),
                           dp = sdesc(base + L::P, 16, 1024);
            const bool tail = ragged && c == chunks - 1;
            wait(&bar.ready, c & 1, dead);
            if (outs) {
                if (c > 0) wait(&bar.o_free, (c - 1) & 1, dead);
                tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)  // (Q S)^T
                        mma_ts(tmem + TM_O1, tmem + TM_S + 8 * k, desc_plus(dq, (k >> 2) * L::panel + (k & 3) * 32), kTS, k > 0);
                }
                __syncwarp();
                wait(&bar.p_ready, c & 1, dead);
            }
            if (tail) wait(&bar.fixed, 0, dead);
            tc_fence_after();
            if (outs) {
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // (P V)^T
                        mma_bf16(tmem + TM_O2, desc_plus(dv, k * 2048), desc_plus(dp, k * 32), kPV, k > 0);
                    mma_commit(smem_u32(&bar.o_done));
                }
                __syncwarp();
                if (c + 1 < chunks) scores(c + 1);
            }
            if (elect()) {
#pragma unroll
                for (int k = 0; k < 4 * kParts; ++k)  // (K^T V~)^T
                    mma_ts(tmem + TM_D, tmem + TM_V + 32 * (k >> 2) + 8 * (k & 3), desc_plus(dk, (k & 3) * 2048), kTD, k > 0);
                mma_commit(smem_u32(&bar.d_done));
                mma_commit(smem_u32(&bar.empty[c % kStages]));
            }
            __syncwarp();
        }
        wait(&bar.d_done, (chunks - 1) & 1, dead);
    } else {
        // ---- the copies, and the gates: two tokens a lane, sums in fixed point
        auto copies = [&](int c) {
            const int i = c % kStages, row = sq.begin + (c_first + c) * kChunk;
            if (elect()) {
                const uint32_t at = smem_u32(smem + i * L::stage), full = smem_u32(&bar.full[i]);
                const int vt = (nv + 63) / 64;
                mbar_expect_tx(full, (NP * (outs ? 2 : 1) + vt) * T8);
                for (int p = 0; p < NP; ++p) {
                    tma_load_3d(at + p * L::panel + T8, &mk, 64 * p, h / a.hdiv, row, full);
                    if (outs) tma_load_3d(at + p * L::panel, &mq, 64 * p, h / a.hdiv, row, full);
                }
                for (int p = 0; p < vt; ++p) tma_load_3d(at + L::V + p * T8, &mv, v0 + 64 * p, h, row, full);
            }
            __syncwarp();
        };
        int64_t total = 0;
        auto load = [&](int c, float* g) {
            const int64_t t = int64_t(c_first + c) * kChunk + 2 * lane;
#pragma unroll
            for (int u = 0; u < 2; ++u) g[u] = t + u < sq.len ? __ldg(a.g + (sq.begin + t + u) * a.gs + h) : 0.f;
        };
        float next[2];
        load(0, next);
        bool lost = false;  // a NaN among the gates
        for (int c = 0; c < chunks; ++c) {
            if (c >= kStages) wait(&bar.empty[c % kStages], ((c / kStages) - 1) & 1, dead);
            copies(c);
            float g[2] = {next[0], next[1]};
            if (c + 1 < chunks) load(c + 1, next);
            const unsigned n0 = __ballot_sync(kFull, g[0] != g[0]), n1 = __ballot_sync(kFull, g[1] != g[1]);
            // a NaN's token and all after it
            const int nan = min(n0 ? 2 * (__ffs(n0) - 1) : 64, n1 ? 2 * __ffs(n1) - 1 : 64);
            int64_t b[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) b[u] = __float2ll_rn(fminf(fmaxf(g[u], -kForget), kForget) * kFixed);
            b[1] += b[0];
            int64_t ps = b[1];
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int64_t x = __shfl_up_sync(kFull, ps, s);
                if (lane >= s) ps += x;
            }
            b[0] += ps - b[1], b[1] = ps;
            const int64_t end = __shfl_sync(kFull, ps, 31), mid = __shfl_sync(kFull, ps, 15);
            const float unit = 1.f / kFixed, bad = __int_as_float(0x7fffffff);
            float* to = reinterpret_cast<float*>(smem + L::GATES + (c % kGateRing) * kGateBytes);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = 2 * lane + u;
                const bool x = t >= nan;
                to[kOut + t] = x ? bad : a.scale * expf(__ll2float_rn(b[u]) * unit);
                to[kDec + t] = nan < 64 ? bad : expf(__ll2float_rn(end - b[u]) * unit);
                to[kLocal + t] = x ? bad : __ll2float_rn(b[u] - (t < kSub ? 0 : mid)) * unit;
                if (t < kSub) to[kCross + t] = nan < kSub ? bad : expf(__ll2float_rn(mid - b[u]) * unit);
            }
            if (lane == 0) {
                const float e = __ll2float_rn(end) * unit;
                const bool near = e > -0.7f && e < 0.7f && nan == 64;
                to[kEnd] = nan < 64 ? bad : near ? expm1f(e) : expf(e);
                to[kNear] = near ? 1.f : 0.f;
            }
            warp_arrive(&bar.gates[c % kGateRing], lane);
            total += end;
            total = total < -(int64_t(1) << 60) ? -(int64_t(1) << 60) : total > (int64_t(1) << 60) ? (int64_t(1) << 60) : total;
            lost |= nan < 64;
        }
        for (int c = max(0, chunks - kStages); c < chunks; ++c) wait_full(c);  // every copy has come before the CTA ends
        if (kPart == Part::first && lane == 0 && v0 == 0)
            seg.fades[segment_at(a, seg, si, h, j)] = lost ? __int_as_float(0x7fffffff) : expf(__ll2float_rn(total) * (1.f / kFixed));
    }
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

__global__ void read_flag_kernel(int* out, int clear) {
    *out = g_timeout_flag;
    if (clear) g_timeout_flag = 0;
}

rm_status fail(const char* what, bool map) {
    char msg[256];
    if (map) std::snprintf(msg, sizeof(msg), "linear attention with a carried state: no tensor map for %s (CUresult %d)", what, last_map_result());
    else std::snprintf(msg, sizeof(msg), "linear attention with a carried state: %s failed: %s", what, cuda_error_text());
    return api_fail(RM_ERR_CUDA, msg);
}

// Segments of the longest sequence (1: not cut), and their chunks: as many as keep each launch's CTAs on the GPU's
// 152 multiprocessors at once, of four chunks or more.
int segments(const Args& a, int* chunks) {
    const int all = (a.max_len + kChunk - 1) / kChunk, blocks = (a.Dv + 127) / 128;
    int n = 1 + int(152 / (int64_t(a.H) * blocks * a.S));
    n = n < kMostSegments ? n : kMostSegments;
    n = n < all / 4 ? n : all / 4;
    if (n < 4) return 1;
    *chunks = (all + n - 1) / n;
    return (all + *chunks - 1) / *chunks;
}

template <int DK>
rm_status launch(const Args& a, rm_dtype state_dt, cudaStream_t s) {
    CUtensorMap mq, mk, mv, mo;
    const int64_t ostr[2] = {int64_t(a.H) * a.Dv, a.Dv};
    if (!map_of(&mq, a.q, DK, a.H / a.hdiv, a.N, a.qs)) return fail("q", true);
    if (!map_of(&mk, a.k, DK, a.H / a.hdiv, a.N, a.ks)) return fail("k", true);
    if (!map_of(&mv, a.v, a.Dv, a.H, a.N, a.vs)) return fail("v", true);
    if (!map_of(&mo, a.o, a.Dv, a.H, a.N, ostr)) return fail("o", true);
    Segments seg{0, 1, nullptr, nullptr};
    const int segs = segments(a, &seg.chunks);
    const unsigned blocks = unsigned((a.Dv + 127) / 128);
    auto walk = [&](auto f, dim3 grid) {
        if (!set_smem(f, WalkSmem<DK>::bytes)) return fail("shared-memory attribute of the walk", false);
        f<<<grid, kWalkThreads, WalkSmem<DK>::bytes, s>>>(a, seg, mq, mk, mv, mo);
        note_launch(1);
        return launch_ok() ? RM_OK : fail("launch of the walk", false);
    };
    const bool f = state_dt == RM_F32;
    if (segs == 1)
        return f ? walk(gla_walk_kernel<DK, float, Part::whole>, dim3(blocks * a.H, a.S))
                 : walk(gla_walk_kernel<DK, __nv_bfloat16, Part::whole>, dim3(blocks * a.H, a.S));
    seg.most = segs;
    seg.ends = static_cast<float*>(a.ws);
    seg.fades = seg.ends + int64_t(a.S) * a.H * segs * a.Dk * a.Dv;
    const dim3 grid(blocks * a.H, a.S, segs - 1);
    const rm_status st = f ? walk(gla_walk_kernel<DK, float, Part::first>, grid) : walk(gla_walk_kernel<DK, __nv_bfloat16, Part::first>, grid);
    if (st != RM_OK) return st;
    return f ? walk(gla_walk_kernel<DK, float, Part::rest>, grid) : walk(gla_walk_kernel<DK, __nv_bfloat16, Part::rest>, grid);
}

}  // namespace

bool tc_supports(const Args& a, rm_dtype dt) {
    return !a.recurrent && dt == RM_BF16 && (a.Dk == 64 || a.Dk == 128) && a.max_len >= kChunkedLen && a.H <= 65535;
}

// A smaller problem may be cut into more segments than this one, so the bound is that of all of them: with n >= 4
// segments heads x sequences x (n - 1) <= 152, so heads x sequences x n <= 152 + 152 / 3 = 202.
size_t tc_workspace_bytes(const Args& a) { return size_t(kMostStates) * (size_t(a.Dk) * a.Dv + 1) * sizeof(float) + 16; }

rm_status tc_launch(const Args& a, rm_dtype state_dt, cudaStream_t s) {
    return a.Dk == 64 ? launch<64>(a, state_dt, s) : launch<128>(a, state_dt, s);
}

}  // namespace gla

rm_status glatc_read_timeout_flag(int* host_flag, int clear, int* dev_scratch, cudaStream_t s) {
    gla::read_flag_kernel<<<1, 1, 0, s>>>(dev_scratch, clear);
    if (!launch_ok()) return RM_ERR_CUDA;
    note_launch(1);
    if (cudaMemcpyAsync(host_flag, dev_scratch, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return RM_ERR_CUDA;
    return cudaStreamSynchronize(s) == cudaSuccess ? RM_OK : RM_ERR_CUDA;
}

}  // namespace rmcp
