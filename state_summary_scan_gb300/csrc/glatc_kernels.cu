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
// nearest, with no run of accumulations.  The decays within a chunk are formed from differences of running sums held in
// two floats, between tokens of one block of 16 directly and between blocks through the blocks' ends, so that with gates of at
// most 0 no factor but e^{-b} within a block (which is not used where it would be large) is above 1.
//
// Where the sequences and heads are too few to fill the GPU, long sequences are cut into segments.  A segment's
// map of the state is S -> e^{sum g} S + dS: a first launch walks the first segment, and the inner ones from zero
// without outputs; gla_compose_kernel carries the states from segment to segment, and a second walk takes the segments
// after the first from them.
//
// A chunk passes through groups of warps with barriers of their own: V~ (eight warps: fragments of V by ldmatrix, times the
// decays, split, into tensor memory), the state (eight), the scores (four), the outputs (four), two that issue products,
// one of which copies too, two of gates.  The code of all of them together has to stay small: with loops unrolled
// the warps wait for instructions (a chunk took 6700 cycles at first, 94 KB of code).  A chunk and head takes 1.25 to 1.55 us now,
// which with 152 equal heads is HBM's rate (one prompt of 8192: 192 us, 6.6 TB/s); with fewer, what bounds it is the loop scores -> P -> P V -> scores and the outputs' way out of tensor memory, which has no room for a second
// set of accumulators, with issue at 55% and the tensor pipe at 36%.  13 ragged prompts of up to 4096 tokens, 32 heads of 128 x 128,
// bf16 pool: 121 us, 4.6 TB/s of what the call cannot do without; one prompt of 8192, 16 heads: 58 us.
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
using gds::warp_arrive;
using gds::zero_rows;

namespace {

constexpr float kForget = 110.f;             // e^-110 is 0 in fp32: lower gates are raised to -110
constexpr int kMostSegments = 32;
constexpr int kMostStates = 320;             // of segments: see tc_workspace_bytes()

// A chunk's gates in shared memory, in floats.  Decays between tokens of one block of 16 are formed from their
// distances in it, those between blocks through the blocks' ends.
constexpr int kSub = 16;
constexpr int kOut = 0;      // scale e^{b_t}
constexpr int kDec = 64;     // e^{b_63 - b_t}
constexpr int kLocal = 128;  // b_t from the start of its block
constexpr int kBack = 192;   // e^{-that}
constexpr int kCross = 256;  // e^{(b at the block's end) - b_t}
constexpr int kEnd = 320;    // the state's decay: S + kEnd S (kNear), or kEnd S
constexpr int kNear = 321;
constexpr int kWeak = 322;   // every |b_t| from the start of its block is below kWeakLimit: e^{b_t - b_s} as a product
constexpr float kWeakLimit = 60.f;
constexpr int kBlocks = 324; // [3] e^{sum of the gates of block 1}, of blocks 1 and 2, of block 2: the decays over blocks between
constexpr uint32_t kGateBytes = 1408;
constexpr int kGateRing = 4;
constexpr int kStages = 4;
constexpr int kAhead = 2;  // chunks whose copies are under way: into stages that were left a chunk ago, so that no copy waits
constexpr int kGroups = 2;  // groups of four warps of the state, and of V~
// then four warps of outputs, four of scores, two of products (the first makes the copies too), two of gates
constexpr int kValueWarp = 4 * kGroups, kOutWarp = 2 * kValueWarp, kScoreWarp = kOutWarp + 4, kMmaWarp = kScoreWarp + 4, kGateWarp = kMmaWarp + 2, kGateWarps = 2;
constexpr int kWalkThreads = (kGateWarp + kGateWarps) * 32;
// Registers a thread: at the launch, and then those of the state's warps and of all others, whose sum is the launch's
constexpr int kLaunchRegisters = 65536 / kWalkThreads / 8 * 8, kStateRegisters = 112, kOtherRegisters = 56;
static_assert(32 * kValueWarp * kStateRegisters + (kWalkThreads - 32 * kValueWarp) * kOtherRegisters <= kWalkThreads * kLaunchRegisters,
              "more registers than the launch has: setmaxnreg.inc would wait for them without end");
static_assert(kValueWarp % 4 == 0, "setmaxnreg is for warpgroups");
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <int DK>
struct WalkSmem {
    static constexpr int NP = DK / 64;
    // a stage: for each 64 dimensions 64 rows of Q, then 64 of K; then V
    static constexpr uint32_t panel = 2 * T8, V = NP * panel, stage = V + 2 * T8;
    static constexpr uint32_t P = kStages * stage, OUT = P + T8, GATES = OUT + 2 * T8;
    static constexpr size_t bytes = GATES + kGateRing * kGateBytes + 1024;
};
static_assert(WalkSmem<128>::bytes <= 227 * 1024, "shared memory of a CTA");

// Tensor-memory columns: K^T V~ transposed, scores, Q S and P V transposed (fp32), then S^T and V~^T (bf16 pairs; of a
// half of the tokens its parts)
constexpr uint32_t TM_D = 0, TM_SC = 128, TM_O1 = 192, TM_O2 = 256, TM_S = 320, TM_V = 384;

struct WalkBars {
    uint64_t full[kStages], empty[kStages], gates[kGateRing], gates_free[kGateRing];
    uint64_t v_free[kGroups];  // a group's half of V~ has been used
    uint64_t d_ready;          // V~ is there, and K^T V~ of the chunk before has been read
    uint64_t o1_ready;         // S is there, and the outputs of the chunk before have been read
    uint64_t scores, p_ready, d_done, o1_done, o_done, fixed;
};

enum class Part { whole, first, rest };  // as the delta rule's walk divides the sequences (gdstc_kernels.cu)
struct Segments {
    int first;     // chunks of a sequence's first segment, at most those of the others
    int chunks;    // of each other segment
    int most;      // segments of the longest sequence
    float* ends;   // [S][H][most][Dk][Dv]: dS of the inner segments, the first one's end
    float* fades;  // [S][H][most]: e^{sum g}
    __device__ __forceinline__ int begin(int j) const { return j == 0 ? 0 : first + (j - 1) * chunks; }
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

// A converged warp's bounded wait, in few instructions (the warps' loops together fill the instruction cache): a
// poll suspends the warp for a microsecond at most, 2^18 of them end it; after one that ran out its others give up soon.
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, uint32_t& polls) {
    const uint32_t b = smem_u32(bar);
    for (uint32_t i = 0; i < polls; ++i) {
        uint32_t ok;
        asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\nselp.u32 %0, 1, 0, p;\n}\n"
                     : "=r"(ok) : "r"(b), "r"(parity) : "memory");
        if (ok) {
            __syncwarp();
            return;
        }
    }
    atomicExch(&g_timeout_flag, 1);
    polls = 16;
}

// A sum held as two floats, to some 2^-48 of its terms
struct Sum2 {
    float hi, lo;
};
__device__ __forceinline__ Sum2 sum2(Sum2 x, Sum2 y) {
    const float s = x.hi + y.hi, z = s - x.hi, e = (x.hi - (s - z)) + (y.hi - z);
    return Sum2{s, e + (x.lo + y.lo)};
}
__device__ __forceinline__ float operator-(Sum2 x, Sum2 y) { return (x.hi - y.hi) + (x.lo - y.lo); }

// The upper halves of a pair as bf16, and the pair less them (exactly)
__device__ __forceinline__ uint32_t cut2(uint64_t& y) {
    uint32_t y0, y1;
    unpair(y, y0, y1);
    y = sub2(y, pair(y0 & 0xffff0000u, y1 & 0xffff0000u));
    return __byte_perm(y0, y1, 0x7632);
}

// Four 8 x 8 tiles of 16-bit elements, transposed: lane i gives the address of row i % 8 of tile i / 8, and has
// column i / 4 of each tile, rows 2 (i % 4) and the next.
__device__ __forceinline__ void ldmatrix_t(uint32_t at, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void stmatrix_t(uint32_t at, const uint32_t* r) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// The same fragments in tensor memory, 16 lanes: eight words of them (two tiles above one another, twice)
__device__ __forceinline__ void tmem_st_16x128(uint32_t at, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// and 16 columns of fp32: pairs of columns 2 (i % 4) .. of lanes i / 4 and i / 4 + 8, for each eight columns
__device__ __forceinline__ void tmem_ld_16x256(uint32_t at, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
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
    __shared__ float sum_s[kGateWarps];
    __shared__ int lost_s[kGateWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blocks = (a.Dv + 127) / 128;
    const int h = blockIdx.x / blocks, v0 = blockIdx.x % blocks * 128, nv = min(a.Dv - v0, 128);
    const int si = kPart == Part::whole ? by_length(a, blockIdx.y) : int(blockIdx.y);
    const Seq sq = sequence(a, si);
    const int all = (sq.len + kChunk - 1) / kChunk;  // the sequence's chunks
    const int j = kPart == Part::whole ? 0 : int(blockIdx.z) + (kPart == Part::rest ? 1 : 0);
    const int c_first = kPart == Part::whole ? 0 : seg.begin(j);
    // the sequence's last segment (the last one that there is takes what a sequence has beyond max_len)
    const bool ends = kPart == Part::whole || j == seg.most - 1 || seg.begin(j + 1) >= all;
    const int chunks = (ends ? all : seg.begin(j + 1)) - c_first;
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
            mbar_init(smem_u32(&bar.empty[i]), (outs ? 2 : 1) + quads * kGroups);
        }
        for (int i = 0; i < kGateRing; ++i) {
            mbar_init(smem_u32(&bar.gates[i]), 1);
            // a chunk's gates are free when the state's warps have seen its K^T V~, for which V~'s warps have read them, and the
            // outputs' warps its outputs, for which the scores' have
            mbar_init(smem_u32(&bar.gates_free[i]), quads * (kGroups + (outs ? 1 : 0)));
        }
        for (int i = 0; i < kGroups; ++i) mbar_init(smem_u32(&bar.v_free[i]), 1);
        mbar_init(smem_u32(&bar.d_ready), 2 * quads * kGroups);
        mbar_init(smem_u32(&bar.o1_ready), quads * (kGroups + 1));
        mbar_init(smem_u32(&bar.scores), 1);
        mbar_init(smem_u32(&bar.p_ready), 4);
        mbar_init(smem_u32(&bar.d_done), 1);
        mbar_init(smem_u32(&bar.o1_done), 1);
        mbar_init(smem_u32(&bar.o_done), 1);
        mbar_init(smem_u32(&bar.fixed), quads * kGroups);
        mbar_fence_init();
    }
    if (warp == 0) tmem_alloc(smem_u32(&tmem_slot), 512);
    // P: what lies above the diagonal's blocks stays zero
    for (int i = tid; i < int(T8) / 16; i += kWalkThreads) *reinterpret_cast<uint4*>(smem + L::P + i * 16) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    uint32_t polls = 1u << 18;
    auto gates_of = [&](int c) {  // the chunk's gates, once they are there
        wait(&bar.gates[c % kGateRing], (c / kGateRing) & 1, polls);
        return reinterpret_cast<const float*>(smem + L::GATES + (c % kGateRing) * kGateBytes);
    };
    auto wait_full = [&](int c) { wait(&bar.full[c % kStages], (c / kStages) & 1, polls); };

    if (warp < kValueWarp) {
        // ---- the state: a lane is a value column, a group has half of its rows
        more_registers<kStateRegisters>();
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
                } else {  // the end of the segment before
                    const float* e = seg.ends + segment_at(a, seg, si, h, j - 1) * DK * a.Dv + v0 + row;
                    rows([&](int r) { return e[int64_t(r) * a.Dv]; });
                }
            }
            warp_arrive(&bar.d_ready, lane);
            for (int c = 0;; ++c) {
                if (c > 0) {  // S <- e^{b_63} S + K^T V~ of the chunk before
                    const float* gates = gates_of(c - 1);
                    const uint64_t end = pair(gates[kEnd], gates[kEnd]);
                    const bool near = gates[kNear] != 0.f;
                    wait(&bar.d_done, (c - 1) & 1, polls);
                    warp_arrive(&bar.gates_free[(c - 1) % kGateRing], lane);  // (V~ of that chunk is in the product: its decays have been read)
                    tc_fence_after();
#pragma unroll
                    for (int i0 = 0; i0 < GC / 2; i0 += 8) {
                        uint32_t d[16];
                        tmem_ld<16>(tl + TM_D + r0 + 2 * i0, d);
                        arrived<16>(d);
                        if (i0 + 8 == GC / 2) {
                            tc_fence_before();
                            warp_arrive(&bar.d_ready, lane);
                        }
                        if (near) {  // near 1 the decay's distance from 1 is what is known to all its bits
#pragma unroll
                            for (int i = 0; i < 8; ++i) S[i0 + i] = add2(fma2(end, S[i0 + i], pair(d[2 * i], d[2 * i + 1])), S[i0 + i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) S[i0 + i] = fma2(end, S[i0 + i], pair(d[2 * i], d[2 * i + 1]));
                        }
                    }
                }
                if (c == chunks) break;
                if (outs) {  // S rounded, as an operand
                    if (c > 0) {
                        wait(&bar.o1_done, (c - 1) & 1, polls);
                        tc_fence_after();
                    }
                    uint32_t x[GC / 2];
#pragma unroll
                    for (int i = 0; i < GC / 2; ++i) x[i] = pack2(S[i]);
                    tmem_st<GC / 2>(tl + TM_S + r0 / 2, x);
                    tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(&bar.o1_ready, lane);
                }
            }
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
    } else if (warp < kOutWarp) {
        // ---- V~: a group has half of a chunk's tokens
        fewer_registers<kOtherRegisters>();
        if ((warp & 3) < quads) {
            const int grp = (warp - kValueWarp) >> 2;
            const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16) + TM_V + kParts * (GT / 2) * grp;
            // values come as fragments of 8 x 8: this lane has pairs of tokens 2 (lane % 4) .. of columns lane / 4 .. + 8 m
            const int tok = GT * grp + 2 * (lane & 3);
            uint32_t from[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                from[i] = smem_u32(smem) + L::V + sw_chunk(64, GT * grp + (lane >> 4) * 8 + (lane & 7), 4 * (warp & 3) + 2 * i + ((lane >> 3) & 1));
            for (int c = 0; c < chunks; ++c) {
                const uint32_t stage = (c % kStages) * L::stage;
                const float* gates = gates_of(c);
                wait_full(c);
                if (ragged && c == chunks - 1) {  // keys and values past the sequence's end are other tokens': they must not meet a zero as NaN
                    const int at = (grp * quads + (warp & 3)) * 32 + lane, threads = 32 * quads * kGroups;
#pragma unroll 1
                    for (int p = 0; p < NP; ++p) zero_rows(smem + stage + p * L::panel + T8, 1, last, at, threads);
                    zero_rows(smem + stage + L::V, 2, last, at, threads);
                    fence_async_smem();
                    warp_arrive(&bar.fixed, lane);
                    wait(&bar.fixed, 0, polls);
                }
                if (c > 0) wait(&bar.v_free[grp], (c - 1) & 1, polls);
                tc_fence_after();
#pragma unroll 1
                for (int u = 0; u < GT / 16; ++u) {
                    uint32_t v[2][4];
                    uint64_t w[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        ldmatrix_t(from[i] + stage + u * 2048, v[i]);
                        w[i] = *reinterpret_cast<const uint64_t*>(gates + kDec + tok + 16 * u + 8 * i);
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t x[kParts][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint64_t y = mul2(widen2(v[half][i]), w[i >> 1]);
                            x[0][i] = cut2(y);
                            if (kParts == 3) x[1][i] = cut2(y);
                            x[kParts - 1][i] = pack2(y);
                        }
#pragma unroll
                        for (int p = 0; p < kParts; ++p) tmem_st_16x128(tl + (uint32_t(16 * half) << 16) + GT / 2 * p + 8 * u, x[p]);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&bar.d_ready));
                    mbar_arrive(smem_u32(&bar.empty[c % kStages]));
                }
            }
        }
    } else if (warp < kScoreWarp) {
        // ---- the outputs: a lane is a value column; whole chunks leave as tiles, the last one by rows
        fewer_registers<kOtherRegisters>();
        const int w = warp & 3;
        if (outs && w < quads) {
            const uint32_t tl = tmem + (uint32_t(32 * w) << 16);
            uint8_t* tile = smem + L::OUT;
            const uint32_t to = smem_u32(tile);
            uint32_t half_off[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) half_off[i] = sw_chunk(64, (lane >> 4) * 8 + (lane & 7), 4 * w + 2 * i + ((lane >> 3) & 1));
            warp_arrive(&bar.o1_ready, lane);
            for (int c = 0; c < chunks; ++c) {
                const float* gates = gates_of(c);
                // the store of the chunk before has read the staging
                if (warp == kOutWarp && lane == 0) bulk_wait_read();
                asm volatile("bar.sync 1, %0;" ::"r"(32 * quads) : "memory");
                wait(&bar.o_done, c & 1, polls);
                tc_fence_after();
#pragma unroll 1
                for (int t0 = 0; t0 < kChunk; t0 += 16) {  // 16 tokens of 32 columns, as fragments of 8 x 8
                    uint32_t p[2][16];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        tmem_ld_16x256(tl + (uint32_t(16 * half) << 16) + TM_O1 + t0, p[half]);
                        tmem_ld_16x256(tl + (uint32_t(16 * half) << 16) + TM_O2 + t0, p[half] + 8);
                    }
                    uint64_t f[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) f[u] = *reinterpret_cast<const uint64_t*>(gates + kOut + t0 + 8 * u + 2 * (lane & 3));
                    arrived<16>(p[0]);
                    arrived<16>(p[1]);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t y[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            y[u] = pack2(fma2(f[u >> 1], pair(p[half][2 * u], p[half][2 * u + 1]), pair(p[half][8 + 2 * u], p[half][9 + 2 * u])));
                        stmatrix_t(to + half_off[half] + t0 * 128, y);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {  // the accumulators and the gates have been read
                    mbar_arrive(smem_u32(&bar.o1_ready));
                    mbar_arrive(smem_u32(&bar.gates_free[c % kGateRing]));
                }
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
        // ---- the scores: a warp has a block of 16 rows, in fragments of 8 x 8: rows lane / 4 and + 8, pairs of columns
        // 2 (lane % 4) ..
        fewer_registers<kOtherRegisters>();
        if (outs) {
            const int block = warp & 3, row = lane >> 2, col = 2 * (lane & 3);
            const uint32_t tl = tmem + (uint32_t(32 * block) << 16) + TM_SC;
            const uint32_t to = smem_u32(smem) + L::P + (16 * block + ((lane >> 3) & 1) * 8 + (lane & 7)) * 128;
            for (int c = 0; c < chunks; ++c) {
                const float* gates = gates_of(c);
                wait(&bar.scores, c & 1, polls);
                tc_fence_after();
                const float b0 = gates[kLocal + 16 * block + row], b1 = gates[kLocal + 16 * block + row + 8];
                const float f0 = a.scale * __expf(b0), f1 = a.scale * __expf(b1);
                const bool weak = gates[kWeak] != 0.f;
#pragma unroll 1
                for (int j = 0; j <= block; ++j) {
                    uint32_t x[8], y[4];
                    tmem_ld_16x256(tl + 16 * j, x);
                    arrived<8>(x);
                    if (j < block || weak) {
                        const float m = block - j < 2 ? 1.f : gates[kBlocks + (j == 1 ? 2 : block - 2)];
                        const float* w = gates + (j < block ? kCross : kBack) + 16 * j + col;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint64_t v = mul2(*reinterpret_cast<const uint64_t*>(w + 8 * u), pair(m, m));
                            y[2 * u] = pack2(mul2(mul2(pair(f0, f0), pair(x[4 * u], x[4 * u + 1])), v));
                            y[2 * u + 1] = pack2(mul2(mul2(pair(f1, f1), pair(x[4 * u + 2], x[4 * u + 3])), v));
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float2 b = *reinterpret_cast<const float2*>(gates + kLocal + 16 * j + 8 * u + col);
                            y[2 * u] = pack2(a.scale * __uint_as_float(x[4 * u]) * __expf(b0 - b.x), a.scale * __uint_as_float(x[4 * u + 1]) * __expf(b0 - b.y));
                            y[2 * u + 1] = pack2(a.scale * __uint_as_float(x[4 * u + 2]) * __expf(b1 - b.x), a.scale * __uint_as_float(x[4 * u + 3]) * __expf(b1 - b.y));
                        }
                    }
                    if (j == block) {  // tokens after the row's own are not seen, whatever they hold
                        const uint32_t own = col < row ? 0xffffffffu : col == row ? 0xffffu : 0u;
                        y[0] &= own, y[2] = 0, y[3] &= own;
                    }
                    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(to + (((2 * j + (lane >> 4)) ^ (lane & 7)) << 4)),
                                 "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                                 : "memory");
                }
                tc_fence_before();
                fence_async_smem();
                warp_arrive(&bar.p_ready, lane);  // P is there, and the scores have been read
            }
        }
    } else {
        fewer_registers<kOtherRegisters>();  // (one instruction for every warp of a warpgroup: different ones are undefined)
        if (warp == kMmaWarp) {
            // ---- the copies, and the products of the state, K^T V~.  The whole warp walks the loop and one elected lane issues.
            const uint32_t base = smem_u32(smem);
            constexpr uint32_t kTD = idesc_bf16(128, DK, 0, 1);
            auto copies = [&](int c) {
                const int i = c % kStages, row = sq.begin + (c_first + c) * kChunk;
                if (c >= kStages) wait(&bar.empty[i], ((c / kStages) - 1) & 1, polls);
                if (elect()) {
                    const uint32_t at = base + i * L::stage, full = smem_u32(&bar.full[i]);
                    const int vt = (nv + 63) / 64;
                    mbar_expect_tx(full, (NP * (outs ? 2 : 1) + vt) * T8);
    #pragma unroll 1
                    for (int p = 0; p < NP; ++p) {
                        tma_load_3d(at + p * L::panel + T8, &mk, 64 * p, h / a.hdiv, row, full);
                        if (outs) tma_load_3d(at + p * L::panel, &mq, 64 * p, h / a.hdiv, row, full);
                    }
    #pragma unroll 1
                    for (int p = 0; p < vt; ++p) tma_load_3d(at + L::V + p * T8, &mv, v0 + 64 * p, h, row, full);
                }
                __syncwarp();
            };
    #pragma unroll 1
            for (int c = 0; c < min(chunks, kAhead); ++c) copies(c);
            for (int c = 0; c < chunks; ++c) {
                if (c + kAhead < chunks) copies(c + kAhead);
                const uint64_t dk = sdesc(base + (c % kStages) * L::stage + T8, L::panel, 1024);
                wait_full(c);
                if (ragged && c == chunks - 1) wait(&bar.fixed, 0, polls);
                wait(&bar.d_ready, c & 1, polls);
                tc_fence_after();
                if (elect()) {
    #pragma unroll 1
                    for (int half = 0; half < kGroups; ++half) {
    #pragma unroll
                        for (int k = 0; k < 2 * kParts; ++k)  // the parts of V~ on 32 tokens
                            mma_ts(tmem + TM_D, tmem + TM_V + kParts * 16 * half + 8 * k, desc_plus(dk, half * 4096 + (k & 1) * 2048), kTD, half + k > 0);
                        mma_commit(smem_u32(&bar.v_free[half]));
                    }
                    mma_commit(smem_u32(&bar.d_done));
                    mma_commit(smem_u32(&bar.empty[c % kStages]));
                }
                __syncwarp();
            }
            wait(&bar.d_done, (chunks - 1) & 1, polls);  // (every copy has come)
        } else if (warp == kMmaWarp + 1) {
            // ---- the products of the outputs: Q S, P V, and Q K^T of the next chunk
            if (outs) {
                const uint32_t base = smem_u32(smem);
                constexpr uint32_t kSc = idesc_bf16(64, 64, 0, 0), kTS = idesc_bf16(128, 64, 0, 0), kPV = idesc_bf16(128, 64, 1, 0);
                for (int c = -1; c < chunks; ++c) {
                    const uint32_t at = base + (c % kStages) * L::stage;
                    if (c >= 0) {
                        const uint64_t dq = sdesc(at, 16, 1024), dv = sdesc(at + L::V, T8, 1024), dp = sdesc(base + L::P, 16, 1024);
                        if (c + 1 < chunks) wait_full(c + 1);
                        wait(&bar.o1_ready, c & 1, polls);
                        tc_fence_after();
                        if (elect()) {
    #pragma unroll 1
                            for (int p = 0; p < NP; ++p)
    #pragma unroll
                                for (int k = 0; k < 4; ++k)  // (Q S)^T
                                    mma_ts(tmem + TM_O1, tmem + TM_S + 32 * p + 8 * k, desc_plus(dq, p * L::panel + k * 32), kTS, p + k > 0);
                            mma_commit(smem_u32(&bar.o1_done));
                        }
                        __syncwarp();
                        if (ragged && c == chunks - 1) wait(&bar.fixed, 0, polls);
                        wait(&bar.p_ready, c & 1, polls);
                        tc_fence_after();
                        if (elect()) {
    #pragma unroll
                            for (int k = 0; k < 4; ++k)  // (P V)^T
                                mma_bf16(tmem + TM_O2, desc_plus(dv, k * 2048), desc_plus(dp, k * 32), kPV, k > 0);
                            mma_commit(smem_u32(&bar.o_done));
                            mma_commit(smem_u32(&bar.empty[c % kStages]));
                        }
                        __syncwarp();
                    }
                    if (c + 1 < chunks) {  // Q K^T of the next chunk, which may replace this one's: its P has been used
                        const uint32_t next = base + ((c + 1) % kStages) * L::stage;
                        const uint64_t d = sdesc(next, 16, 1024), dk = sdesc(next + T8, 16, 1024);
                        if (c < 0) wait_full(0);
                        tc_fence_after();
                        if (elect()) {
    #pragma unroll 1
                            for (int p = 0; p < NP; ++p)
    #pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_bf16(tmem + TM_SC, desc_plus(d, p * L::panel + k * 32), desc_plus(dk, p * L::panel + k * 32), kSc, p + k > 0);
                            mma_commit(smem_u32(&bar.scores));
                        }
                        __syncwarp();
                    }
                }
                wait(&bar.o_done, (chunks - 1) & 1, polls);
            }
        } else {
            // ---- the gates, two tokens a lane, every other chunk a warp, as far ahead as there is room
            Sum2 total{0.f, 0.f};
            auto load = [&](int c, float* g) {
                const int64_t t = int64_t(c_first + c) * kChunk + 2 * lane;
    #pragma unroll
                for (int u = 0; u < 2; ++u) g[u] = t + u < sq.len && c < chunks ? __ldg(a.g + (sq.begin + t + u) * a.gs + h) : 0.f;
            };
            float next[2];
            load(warp - kGateWarp, next);
            bool lost = false;  // a NaN among the gates
            for (int c = warp - kGateWarp; c < chunks; c += kGateWarps) {
                float g[2] = {next[0], next[1]};
                load(c + kGateWarps, next);
                const unsigned n0 = __ballot_sync(kFull, g[0] != g[0]), n1 = __ballot_sync(kFull, g[1] != g[1]);
                // a NaN's token and all after it
                const int nan = min(n0 ? 2 * (__ffs(n0) - 1) : 64, n1 ? 2 * __ffs(n1) - 1 : 64);
    #pragma unroll
                for (int u = 0; u < 2; ++u) g[u] = fminf(fmaxf(g[u], -kForget), kForget);
                const Sum2 own = sum2(Sum2{g[0], 0.f}, Sum2{g[1], 0.f});
                Sum2 ps = own;
    #pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const Sum2 x{__shfl_up_sync(kFull, ps.hi, s), __shfl_up_sync(kFull, ps.lo, s)};
                    if (lane >= s) ps = sum2(ps, x);
                }
                const Sum2 before = sum2(ps, Sum2{-g[1], 0.f});
                const Sum2 end{__shfl_sync(kFull, ps.hi, 31), __shfl_sync(kFull, ps.lo, 31)};
                // the sums at the end of this lane's block of 16, and before it
                const Sum2 own_end{__shfl_sync(kFull, ps.hi, lane | 7), __shfl_sync(kFull, ps.lo, lane | 7)};
                Sum2 begin{__shfl_sync(kFull, ps.hi, (lane | 7) - 8 & 31), __shfl_sync(kFull, ps.lo, (lane | 7) - 8 & 31)};
                if (lane < 8) begin = Sum2{0.f, 0.f};
                const float bad = __int_as_float(0x7fffffff);
                if (c >= kGateRing) wait(&bar.gates_free[c % kGateRing], ((c / kGateRing) - 1) & 1, polls);
                float* to = reinterpret_cast<float*>(smem + L::GATES + (c % kGateRing) * kGateBytes);
                bool weak = true;
    #pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    const int t = 2 * lane + u;
                    const bool x = t >= nan;
                    const Sum2 bt = u ? ps : before;
                    const float local = bt - begin;
                    weak = weak && fabsf(local) < kWeakLimit;
                    to[kOut + t] = x ? bad : a.scale * __expf(bt.hi + bt.lo);
                    to[kDec + t] = nan < 64 ? bad : __expf(end - bt);
                    to[kLocal + t] = x ? bad : local;
                    to[kBack + t] = __expf(-local);
                    to[kCross + t] = nan <= (t | (kSub - 1)) ? bad : __expf(own_end - bt);
                }
                weak = __all_sync(kFull, weak);
                // (lanes 15 and 23 end blocks 1 and 2; a NaN there reaches the rows by their own sums)
                const Sum2 e0{__shfl_sync(kFull, ps.hi, 7), __shfl_sync(kFull, ps.lo, 7)}, e1{__shfl_sync(kFull, ps.hi, 15), __shfl_sync(kFull, ps.lo, 15)},
                    e2{__shfl_sync(kFull, ps.hi, 23), __shfl_sync(kFull, ps.lo, 23)};
                if (lane < 3) to[kBlocks + lane] = __expf(lane == 0 ? e1 - e0 : lane == 1 ? e2 - e0 : e2 - e1);
                if (lane == 0) {
                    const float e = end.hi + end.lo;
                    const bool near = e > -0.7f && e < 0.7f && nan == 64;
                    to[kEnd] = nan < 64 ? bad : near ? expm1f(e) : expf(e);
                    to[kNear] = near ? 1.f : 0.f;
                    to[kWeak] = weak ? 1.f : 0.f;
                }
                warp_arrive(&bar.gates[c % kGateRing], lane);
                total = sum2(total, end);
                lost |= nan < 64;
            }
            if (kPart == Part::first && lane == 0) {
                sum_s[warp - kGateWarp] = total.hi + total.lo;
                lost_s[warp - kGateWarp] = lost;
            }
        }
    }
    __syncthreads();
    if (kPart == Part::first && tid == 0 && v0 == 0)
        seg.fades[segment_at(a, seg, si, h, j)] = lost_s[0] || lost_s[1] ? __int_as_float(0x7fffffff) : expf(sum_s[0] + sum_s[1]);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// The states at the segments' ends, in their place: S_j = e^{sum g} S_{j-1} + dS_j.  Four elements a thread, all segments, eight
// of which are read at once.  (Folded by each walk for itself the last ones would read all the others': 6 us of 67.)
__global__ void __launch_bounds__(256) gla_compose_kernel(const __grid_constant__ Args a, const Segments seg) {
    const int64_t at = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4, size = int64_t(a.Dk) * a.Dv;
    const int h = blockIdx.y, i = blockIdx.z;
    const Seq sq = sequence(a, i);
    // the segments that end before the sequence's last one
    const int all = (sq.len + kChunk - 1) / kChunk, inner = min((all - 1 - seg.first + seg.chunks) / seg.chunks, seg.most - 1);
    if (at >= size || sq.slot < 0 || inner < 2) return;
    float* e = seg.ends + segment_at(a, seg, i, h, 0) * size + at;
    const float* f = seg.fades + segment_at(a, seg, i, h, 0);
    float4 s = *reinterpret_cast<const float4*>(e);
    constexpr int kBatch = 8;  // segments that are read together
    for (int j0 = 1; j0 < inner; j0 += kBatch) {
        float4 d[kBatch];
        float x[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (j0 + j < inner) d[j] = *reinterpret_cast<const float4*>(e + (j0 + j) * size), x[j] = f[j0 + j];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (j0 + j < inner) {
                s.x = fmaf(x[j], s.x, d[j].x), s.y = fmaf(x[j], s.y, d[j].y), s.z = fmaf(x[j], s.z, d[j].z), s.w = fmaf(x[j], s.w, d[j].w);
                *reinterpret_cast<float4*>(e + (j0 + j) * size) = s;
            }
        }
    }
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

// Segments of the longest sequence (1: not cut), and their chunks: as many as keep each walk's CTAs on the GPU's 152
// multiprocessors at once, of two chunks or more.  A chunk takes some 1.45 us (64 x 64: 1.1), two more launches and the
// states between them some 13; with n segments the chain is two walks of 1 / n of the chunks.  The others are as long as if the
// first were 0.8 of one, and the first gets what they leave: the first walk takes its outputs, and those of no other, so that in
// equal segments the others wait for it.  One prompt of 8192, 32 heads, chunks of the first and of each other segment, us: 24 and 26
// 97.6, 20 and 27 91.4, 12 and 29 95.9; 16 heads: 11 and 13 58.7, 2 and 14 56.7.  (A gate for each token takes as long.)
// us in a CUDA graph, whole / cut:
//     tokens                          512          1024         2048         8192
//     16 heads of 128 x 128           18.9 / 23.0  30.8 / 25.4  53.8 / 32.1  192 / 57
//     32 heads, or two prompts of 16  19.6 / 24.8  31.4 / 33.1  54.6 / 39.6  193 / 91
//     48 heads (4 segments)           20.1 / 27.2  31.9 / 35.1  54.9 / 46.4  193 / 112
//     8 heads of 128 x 256            18.5 / 22.9  30.5 / 24.8  53.8 / 31.2  194 / 55
//     4 heads of 64 x 64              13.9 / 16.2  22.8 / 17.7  40.5 / 19.0  147 / 26
int segments(const Args& a, Segments* seg) {
    const int all = (a.max_len + kChunk - 1) / kChunk, blocks = (a.Dv + 127) / 128;
    int n = 1 + int(152 / (int64_t(a.H) * blocks * a.S));
    n = n < kMostSegments ? n : kMostSegments;
    n = n < all / 2 ? n : all / 2;
    if (int64_t(all) * (n - 2) <= 10 * n) return 1;
    const int c = (5 * all + 5 * n - 2) / (5 * n - 1);  // all / (n - 0.2) and more
    seg->chunks = c;
    seg->first = all % c ? all % c : c;
    return (all + c - 1) / c;
}

template <int DK>
rm_status launch(const Args& a, rm_dtype state_dt, cudaStream_t s) {
    CUtensorMap mq, mk, mv, mo;
    const int64_t ostr[2] = {int64_t(a.H) * a.Dv, a.Dv};
    if (!map_of(&mq, a.q, DK, a.H / a.hdiv, a.N, a.qs)) return fail("q", true);
    if (!map_of(&mk, a.k, DK, a.H / a.hdiv, a.N, a.ks)) return fail("k", true);
    if (!map_of(&mv, a.v, a.Dv, a.H, a.N, a.vs)) return fail("v", true);
    if (!map_of(&mo, a.o, a.Dv, a.H, a.N, ostr)) return fail("o", true);
    Segments seg{0, 0, 1, nullptr, nullptr};
    const int segs = segments(a, &seg);
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
    gla_compose_kernel<<<dim3(unsigned((a.Dk * a.Dv + 1023) / 1024), unsigned(a.H), unsigned(a.S)), 256, 0, s>>>(a, seg);
    note_launch(1);
    if (!launch_ok()) return fail("launch of the composition", false);
    return f ? walk(gla_walk_kernel<DK, float, Part::rest>, grid) : walk(gla_walk_kernel<DK, __nv_bfloat16, Part::rest>, grid);
}

}  // namespace

bool tc_supports(const Args& a, rm_dtype dt) {
    return !a.recurrent && dt == RM_BF16 && (a.Dk == 64 || a.Dk == 128) && a.max_len >= chunked_len(a) && a.H <= 65535;
}

// A smaller problem may be cut into more segments than this one, so the bound is that of all of them: with n >= 3
// segments heads x sequences x (n - 1) <= 152, so heads x sequences x n <= 152 + 152 / 2 = 228.
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
