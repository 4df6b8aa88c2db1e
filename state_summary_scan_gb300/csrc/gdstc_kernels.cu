// gdstc_kernels.cu -- the gated delta rule with a carried state in chunks of 64 tokens on the
// tensor cores (tcgen05 + TMA): ragged prompts in bf16, Dk in {64, 128}, any Dv.
//
// With b_t the running sum of a chunk's gates, Gam[t][r] = e^{b_t - b_r} (r <= t), A[t][r] =
// beta_t (k_t.k_r) Gam[t][r] (r < t), T = (I + A)^{-1} diag(beta) and S the state before the chunk,
// unrolling the recurrence gives (the WY form of the product of I - beta k k^T):
//     D  = T V - T (K o e^b) S,    O = scale (e^b o (Q S) + (mask(Q K^T) o Gam) D)
//     S' = e^{b_63} S + K^T D~,    D~_t = e^{b_63 - b_t} D_t
// Where every |b_t - b_63| < 60 all decays are taken to the chunk's end, with dec_t = e^{b_63 - b_t}
// and S~ = e^{b_63} S, so that nothing between the products but roundings is left to do:
//     T~ = dec o T,   U = T~ V,   W = T~ (K o 1/dec),   P = mask(Q K^T)
//     D~ = U - W S~,   O = scale / dec o (Q S~ + P D~),   S' = S~ + K^T D~
// Chunks of stronger decay, whose factors would leave fp32, take the first form (T~ = T, W = T (K o
// e^b), P = mask(Q K^T) o Gam).
// Two launches:
//   gds_factor_kernel  every (chunk, head) at once: U, P, -W and the decays, which do not depend on
//                      the state, laid out as the walk copies them in
//   gds_walk_kernel    one CTA per (sequence, head, 128 columns of values): the chain over the
//                      sequence's chunks
// Where the sequences and heads are too few to fill the GPU, long sequences are cut into segments.  A
// segment's map of the state is affine, S -> M S + dS: a first walk takes the first segment, and each
// inner one from zero (dS) and from the identity without values (M); gds_compose_kernel then carries
// the states from segment to segment, and a second walk takes the segments after the first from them.
//
// The walk is bound by the latency of its chain: S -> W S -> D~ -> K^T D~ -> S.  It keeps S
// transposed, a value column a lane, so that every step of the chain is a row of tensor memory per
// thread and the rounded S and D go back to tensor memory as A operands, with no transposition and
// no shared memory.  The state itself accumulates in tensor memory in fp32.  The products that do
// not carry the chain (Q S, P D) run in its pauses, issued by a warp of their own, and the outputs
// are read and stored by others.
//
// Rounding: K, Q and V enter as they are; T~ and D~ as the sum of two bf16 (16 significant bits:
// two products with the exact operand), because their errors reach the state undamped; U is fp32.  S, W and P
// are rounded once to bf16: S and W only enter through W S, which is small beside T V, and P only
// through O, which is rounded to bf16 anyway.  In fp64 with these roundings alone (1024 tokens, 4
// heads of 128): state 1.4e-4 off, o 2.4e-3 with its own rounding of 1.7e-3.  Where W S is not small, a state
// ten and more times what one chunk of 48 or 64 tokens writes: state 1e-3 to 2e-3 off, o as before; after 128
// tokens 5e-5 or less.
#include <cstdio>

#include "gds.cuh"

namespace rmcp {
namespace gds {

using namespace tc;

namespace {

constexpr uint32_t T8 = kTileBytes;      // one [64][64] bf16 tile
constexpr uint32_t kGateBytes = 1024;    // the scale of O (weak) or of Q S [64], dec [64], e^{b_63}, weak (1 or 0)
constexpr int kDec = 64, kEnd = 128, kWeak = 129;
constexpr float kForget = -110.f;        // e^{-110} is 0 in fp32: lower gates are raised to it
constexpr int kMostSegments = 12;
constexpr int kMostStates = 152;         // of segments: see tc_workspace_bytes()
constexpr float kWeakLimit = 60.f;       // decays within a chunk that factor through its end

// Factors of a (chunk, head) in the workspace: P, -W (Dk / 64 swizzled tiles), the gates, then
// U in fp32 as [16 groups of 4 tokens][columns][4] for each block of up to 128 value columns, so
// that a lane of the walk reads its column's four tokens at once.
__host__ __device__ constexpr uint32_t u_cols(int Dv) { return Dv >= 128 ? 128u : uint32_t((Dv + 31) / 32 * 32); }
__host__ __device__ constexpr uint32_t u_bytes(int Dv) { return kChunk * 4 * u_cols(Dv); }  // of a block
__host__ __device__ constexpr uint32_t factor_gates(int Dk) { return (1 + Dk / 64) * T8; }
__host__ __device__ constexpr uint32_t factor_u(int Dk) { return factor_gates(Dk) + kGateBytes; }
__host__ __device__ constexpr uint32_t factor_bytes(int Dk, int Dv) {
    return factor_u(Dk) + uint32_t((Dv + 127) / 128) * u_bytes(Dv);
}

// First chunk of sequence i: chunks of different sequences do not meet, since a sequence of n
// tokens from token b has at most floor((b + n) / 64) - floor(b / 64) + 1 of them.
__device__ __forceinline__ int first_chunk(const Args& a, int i) {
    const int b = a.cu ? min(max(__ldg(a.cu + i), 0), a.N) : i * a.each;
    return b / kChunk + i;
}
// The y-th longest of up to 32 sequences, one a lane, so that the longest walks begin first (13 ragged prompts
// of up to 4096 tokens: 208 to 181 us).  With 33 to 128 ragged prompts of 32 heads a call with the longest
// given first takes 2 to 3.5% less (33 of up to 2048 tokens: 804 for 833 us), which is left.  Whole-warp call.
__device__ __forceinline__ int by_length(const Args& a, int y) {
    if (a.cu == nullptr || a.S > 32) return y;
    const int lane = threadIdx.x & 31, i = min(lane, a.S - 1);
    const int b = min(max(__ldg(a.cu + i), 0), a.N), len = lane < a.S ? min(max(__ldg(a.cu + i + 1), b), a.N) - b : -1;
    int rank = 0;
    for (int j = 0; j < a.S; ++j) {
        const int other = __shfl_sync(kFull, len, j);
        rank += other > len || (other == len && j < lane);
    }
    const unsigned m = __ballot_sync(kFull, lane < a.S && rank == y);
    return m ? __ffs(m) - 1 : y;
}
int chunk_slots(const Args& a) { return a.N / kChunk + a.S + 1; }

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t* r);
template <>
__device__ __forceinline__ void tmem_st<16>(uint32_t at, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
template <>
__device__ __forceinline__ void tmem_st<32>(uint32_t at, const uint32_t* r) { tmem_st32(at, r); }
template <>
__device__ __forceinline__ void tmem_st<8>(uint32_t at, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// N consecutive columns of this warp's lanes, valid after tmem_wait_ld()
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t* r);
template <>
__device__ __forceinline__ void tmem_ld<16>(uint32_t at, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}
template <>
__device__ __forceinline__ void tmem_ld<32>(uint32_t at, uint32_t* r) { tmem_ld32_nowait(at, r); }

// D[tmem] (+)= A[tmem] * B[smem]: A's rows are lanes, two bf16 of K a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Zero rows [n, 64) of `tiles` adjacent [64][64] tiles.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int tiles, int n, int tid, int threads) {
    const int each = (kChunk - n) * 8;  // 16-byte units of a tile
    for (int i = tid; i < tiles * each; i += threads)
        *reinterpret_cast<uint4*>(tile + (i / each) * T8 + n * 128 + (i % each) * 16) = make_uint4(0, 0, 0, 0);
}

// A is [64][64] fp32 with the 16-byte units of a row permuted by the row, so that the same unit of
// 16 rows lies in different banks; X is plain, as its columns are read side by side.
__device__ __forceinline__ int a_unit(int r, int u) { return r * 64 + ((u ^ (r & 15)) << 2); }
__device__ __forceinline__ float4 a_row4(const float* A, int r, int u) { return *reinterpret_cast<const float4*>(A + a_unit(r, u)); }
__device__ __forceinline__ float4 x_row4(const float* X, int r, int u) { return *reinterpret_cast<const float4*>(X + r * 64 + 4 * u); }

// R rows of one column of a product: out[i * 64] = f sum_{k < n} l_i[k] b[k * 64], four terms of the
// rows (kA: of A, from row r, unit u0; else of X) at a time.
template <int R, bool kA>
__device__ __forceinline__ void tri_product(const float* M, int r, int u0, const float* b, int n, float* out, float f) {
    float x[R];
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = 0.f;
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
        if (k >= n) break;
        float4 l[R];
#pragma unroll
        for (int i = 0; i < R; ++i) l[i] = kA ? a_row4(M, r + i, u0 + k / 4) : x_row4(M, r + i, u0 + k / 4);
        const float b0 = b[k * 64], b1 = b[(k + 1) * 64], b2 = b[(k + 2) * 64], b3 = b[(k + 3) * 64];
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = fmaf(l[i].w, b3, fmaf(l[i].z, b2, fmaf(l[i].y, b1, fmaf(l[i].x, b0, x[i]))));
    }
#pragma unroll
    for (int i = 0; i < R; ++i) out[i * 64] = f * x[i];
}

// X = (I + A)^{-1} for the strictly lower A, by halves: the four 16 x 16 diagonal blocks by forward
// substitution (a column a lane), then twice the block below the diagonal of a pair,
// X21 = -X22 (A21 X11).  A21 X11 waits in the pair's block above the diagonal, so that nothing but A
// and X is needed; entries above the diagonal are not zero afterwards (those of A's diagonal blocks
// must be).  All 256 threads call it.  A lane takes a column and two or four rows, which shares every
// read of X between the rows and every read of A between the columns.
__device__ __forceinline__ void halves_inverse(const float* A, float* X) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < 2) {
        const int o = 16 * (2 * warp + (lane >> 4)), c = lane & 15;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float y = r == c ? 1.f : 0.f;
#pragma unroll
            for (int k = 0; k < r; k += 4) {
                const float4 l = a_row4(A, o + r, (o + k) / 4);
                y = fmaf(-l.x, x[k], y);  // in order: only the last term waits for the row before
                if (k + 1 < r) y = fmaf(-l.y, x[k + 1], y);
                if (k + 2 < r) y = fmaf(-l.z, x[k + 2], y);
                if (k + 3 < r) y = fmaf(-l.w, x[k + 3], y);
            }
            x[r] = y;
            X[(o + r) * 64 + o + c] = y;
        }
    }
    __syncthreads();
    {  // pairs of 16: four warps each, two rows a lane
        const int o = 32 * (warp >> 2), r = 4 * (warp & 3) + 2 * (lane >> 4), c = lane & 15;
        tri_product<2, true>(A, o + 16 + r, o / 4, X + o * 64 + o + c, 16, X + (o + r) * 64 + o + 16 + c, 1.f);
        __syncthreads();
        tri_product<2, false>(X, o + 16 + r, o / 4 + 4, X + o * 64 + o + 16 + c, 16, X + (o + 16 + r) * 64 + o + c, -1.f);
        __syncthreads();
    }
    {  // the pair of 32, four rows a lane.  The blocks above the diagonals of X11 and X22 hold sums, not
       // zeros: X11's columns 16 .. 31 start at its row 16, and X22's rows below 16 end at its column 16
        const int r = 4 * warp;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            float4 l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) l[i] = a_row4(A, 32 + r + i, k / 4);
            float b0 = X[k * 64 + lane], b1 = X[(k + 1) * 64 + lane], b2 = X[(k + 2) * 64 + lane], b3 = X[(k + 3) * 64 + lane];
            if (k < 16 && lane >= 16) b0 = b1 = b2 = b3 = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = fmaf(l[i].w, b3, fmaf(l[i].z, b2, fmaf(l[i].y, b1, fmaf(l[i].x, b0, x[i]))));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) X[(r + i) * 64 + 32 + lane] = x[i];
        __syncthreads();
        tri_product<4, false>(X, 32 + r, 8, X + 32 + lane, r < 16 ? 16 : 32, X + (32 + r) * 64 + lane, -1.f);
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// The factors of every (chunk, head).  Rows past the sequence's end have beta = 0, zero keys and
// values and a zero row of P, so that they write nothing and read nothing.
// ---------------------------------------------------------------------------
// Shared memory: for each half h of the key dimensions K_h and Q_h side by side (one operand of
// 128 rows), P, A, X.  V comes in over Q, T~ (hi, lo) lies over A, T~ o 1/dec over P, -W over K, each
// when the other is done with.  72 KB and 128 columns of tensor memory: three CTAs an SM.
//
// 32 heads of 128 x 128, 13 ragged prompts of up to 4096 tokens: 270 us.  Its floor is the traffic of
// what it leaves the walk (57 KB a chunk and head, 33 KB of it U) beside its inputs, some 170 us; the
// rest is the time of a CTA's own steps (two product rounds, the inverse, the epilogues), of which
// three CTAs an SM overlap only part.
constexpr uint32_t FA_K = 0, FA_Q = T8, FA_PANEL = 2 * T8, FA_P = 4 * T8, FA_A = 5 * T8, FA_T = FA_A, FA_X = 7 * T8;
constexpr size_t kFactorSmem = 9 * T8 + 1024;

template <int DK>
__global__ void __launch_bounds__(256, 3)
    gds_factor_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap mq,
                      const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    constexpr int NP = DK / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    float* A = reinterpret_cast<float*>(smem + FA_A);
    float* X = reinterpret_cast<float*>(smem + FA_X);
    __shared__ __align__(16) float b_s[kChunk], beta_s[kChunk], gam_s[kChunk], dec_s[kChunk];
    __shared__ __align__(8) uint64_t full, vfull, mbar;
    __shared__ uint32_t tmem_slot;
    __shared__ int weak_s;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = blockIdx.x, h = blockIdx.y;
    // the sequence of this chunk slot: the last one whose first chunk is at or before it
    int lo = 0;
    for (int left = a.S; left > 1;) {  // 32 of them looked at at once
        const int step = (left + 31) / 32, i = lane * step;
        const int before = __popc(__ballot_sync(kFull, i < left && first_chunk(a, lo + min(i, left - 1)) <= c));
        const int skip = max(before - 1, 0) * step;
        lo += skip;
        left = min(step, left - skip);
    }
    const Seq sq = sequence(a, lo);
    const int t0 = (c - first_chunk(a, lo)) * kChunk;
    if (t0 < 0 || t0 >= sq.len || sq.slot < 0) return;
    const int n = min(sq.len - t0, kChunk);  // tokens of the chunk
    const int64_t tok = sq.begin + t0;
    uint8_t* fac = static_cast<uint8_t*>(a.ws) + (int64_t(c) * a.H + h) * factor_bytes(DK, a.Dv);

    float g[2], be[2];  // warp 0: two tokens a lane
    if (warp == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            g[i] = t < n ? __ldg(a.g + (tok + t) * a.gs + h) : 0.f;
            be[i] = t < n ? __ldg(a.beta + (tok + t) * a.bs + h) : 0.f;
        }
        tmem_alloc(smem_u32(&tmem_slot), 128);
    } else if (tid == 32) {
        mbar_init(smem_u32(&full), 1);
        mbar_init(smem_u32(&vfull), 1);
        mbar_init(smem_u32(&mbar), 1);
        mbar_fence_init();
        mbar_expect_tx(smem_u32(&full), 2 * NP * T8);
        for (int p = 0; p < NP; ++p) {
            tma_load_3d(smem_u32(smem + FA_K + p * FA_PANEL), &mk, 64 * p, h / a.hdiv, int(tok), smem_u32(&full));
            tma_load_3d(smem_u32(smem + FA_Q + p * FA_PANEL), &mq, 64 * p, h / a.hdiv, int(tok), smem_u32(&full));
        }
    }
    if (warp == 0) {  // the running sum of the gates
#pragma unroll
        for (int i = 0; i < 2; ++i) g[i] = g[i] < kForget ? kForget : g[i];
        float ps = g[0] + g[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(kFull, ps, o);
            if (lane >= o) ps += x;
        }
        const float end = __shfl_sync(kFull, ps, 31);
        const float b[2] = {ps - g[1], ps};
        const bool weak = __all_sync(kFull, fabsf(b[0] - end) < kWeakLimit && fabsf(b[1] - end) < kWeakLimit);
        float* gates = reinterpret_cast<float*>(fac + factor_gates(DK));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            b_s[t] = b[i];
            beta_s[t] = be[i];
            const float out = expf(weak ? b[i] - end : b[i]), dec = expf(end - b[i]);
            gam_s[t] = out;
            dec_s[t] = weak ? dec : 1.f;
            gates[t] = a.scale * out;
            gates[kDec + t] = dec;
        }
        if (lane == 0) {
            gates[kEnd] = expf(end);
            gates[kWeak] = weak ? 1.f : 0.f;
            weak_s = weak;
        }
    }
    tc_fence_before();
    __syncthreads();  // barriers, tensor memory and the decays are in place
    tc_fence_after();
    const uint32_t tmem = tmem_slot;  // [0,64) K K^T and Q K^T, then W^T; [64,128) U^T
    mbar_wait(smem_u32(&full), 0);
    if (n < kChunk) {
        for (int p = 0; p < NP; ++p) zero_rows(smem + FA_K + p * FA_PANEL, 1, n, tid, 256);
        fence_async_smem();
        __syncthreads();
    }
    uint32_t mph = 0;
    const int vblocks = (a.Dv + 127) / 128;
    // V of a block over Q (whose product is done by then)
    auto load_v = [&](int vb) {
        const int tiles = min((a.Dv - 128 * vb + 63) / 64, 2);
        mbar_expect_tx(smem_u32(&vfull), tiles * T8);
        for (int p = 0; p < tiles; ++p)
            tma_load_3d(smem_u32(smem + FA_Q + p * FA_PANEL), &mv, 128 * vb + 64 * p, h, int(tok), smem_u32(&vfull));
    };
    if (warp == 0) {
        if (elect()) {  // [K; Q] K^T
            const uint64_t d = sdesc(smem_u32(smem + FA_K), 16, 1024);
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                const uint32_t at = (k >> 2) * FA_PANEL + (k & 3) * 32;
                mma_bf16(tmem, desc_plus(d, at), desc_plus(d, at), idesc_bf16(128, 64, 0, 0), k > 0);
            }
            mma_commit(smem_u32(&mbar));
        }
        __syncwarp();
    }
    mbar_wait(smem_u32(&mbar), mph);
    mph ^= 1;
    tc_fence_after();
    if (tid == 0) load_v(0);
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t tl = tmem + (uint32_t(32 * quad) << 16) + 32 * half;
    {
        // rows 0 .. 63 are K's, 64 .. 127 are Q's; this warp's columns r are 32 half ..
        uint32_t x[32];
        tmem_ld<32>(tl, x);
        tmem_wait_ld();
        const int t = 32 * (quad & 1) + lane;
        const float bt = b_s[t];
        // (the decays of a weak chunk factor through its end, and P has none)
        if (quad < 2) {
            const float f = beta_s[t] * (weak_s ? gam_s[t] : 1.f);
            if (quad >= half) {  // the other block lies above the diagonal and is not read
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const int r = 32 * half + e;
                    float4 m;
                    if (weak_s) {
                        m = *reinterpret_cast<const float4*>(dec_s + r);
                    } else {
                        const float4 b = *reinterpret_cast<const float4*>(b_s + r);
                        m = make_float4(__expf(bt - b.x), __expf(bt - b.y), __expf(bt - b.z), __expf(bt - b.w));
                    }
                    float4 y;
                    y.x = r < t ? f * __uint_as_float(x[e]) * m.x : 0.f;
                    y.y = r + 1 < t ? f * __uint_as_float(x[e + 1]) * m.y : 0.f;
                    y.z = r + 2 < t ? f * __uint_as_float(x[e + 2]) * m.z : 0.f;
                    y.w = r + 3 < t ? f * __uint_as_float(x[e + 3]) * m.w : 0.f;
                    *reinterpret_cast<float4*>(A + a_unit(t, r >> 2)) = y;
                }
            }
        } else {
            const int most = t < n ? t : -1;  // the last key that the row sees
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 32 * half + e + i;
                    const float m = weak_s ? 1.f : __expf(bt - b_s[r]);
                    y[i] = r <= most ? __uint_as_float(x[e + i]) * m : 0.f;
                }
                *reinterpret_cast<uint4*>(smem + FA_P + sw_chunk(64, t, (32 * half + e) >> 3)) = pack8(y);
            }
        }
    }
    fence_async_smem();
    __syncthreads();
    if (warp == 0) {
        if (elect()) {
            bulk_store(fac, smem_u32(smem + FA_P), T8);
            bulk_commit();
        }
        __syncwarp();
    }
    halves_inverse(A, X);
    if (warp == 0) {
        if (elect()) bulk_wait_read();  // P has left
        __syncwarp();
    }
    __syncthreads();
    {  // T~, hi and lo, and T~ o 1/dec (or T o e^b) for W: a row at a time, two columns a lane
        const float2 be = *reinterpret_cast<const float2*>(beta_s + 2 * lane), ga = *reinterpret_cast<const float2*>(gam_s + 2 * lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int t = 8 * warp + i;
            const float2 v = *reinterpret_cast<const float2*>(X + t * 64 + 2 * lane);
            const float f = dec_s[t];
            const float x0 = 2 * lane <= t ? v.x * be.x * f : 0.f, x1 = 2 * lane + 1 <= t ? v.y * be.y * f : 0.f;
            const uint32_t at = t * 128 + (((lane >> 2) ^ i) << 4) + (lane & 3) * 4;
            uint32_t high, low;
            split2(pair(x0, x1), high, low);
            *reinterpret_cast<uint32_t*>(smem + FA_T + at) = high;
            *reinterpret_cast<uint32_t*>(smem + FA_T + T8 + at) = low;
            *reinterpret_cast<uint32_t*>(smem + FA_P + at) = pack2(x0 * ga.x, x1 * ga.y);
        }
    }
    for (int vb = 0; vb < vblocks; ++vb) {
        mbar_wait(smem_u32(&vfull), vb & 1);
        if (n < kChunk)
            for (int p = 0; p < 2; ++p) zero_rows(smem + FA_Q + p * FA_PANEL, 1, n, tid, 256);
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 0) {
            if (elect()) {
                const uint64_t dt = sdesc(smem_u32(smem + FA_T), 16, 1024), dv = sdesc(smem_u32(smem + FA_Q), FA_PANEL, 1024);
                if (vb == 0) {  // W^T = K^T (T~ o 1/dec)^T
                    const uint64_t dk = sdesc(smem_u32(smem + FA_K), FA_PANEL, 1024), dg = sdesc(smem_u32(smem + FA_P), 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem, desc_plus(dk, k * 2048), desc_plus(dg, k * 32), idesc_bf16(128, 64, 1, 0), k > 0);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)  // U^T = V^T T~^T
                    mma_bf16(tmem + 64, desc_plus(dv, (k & 3) * 2048), desc_plus(dt, (k >> 2) * T8 + (k & 3) * 32),
                             idesc_bf16(128, 64, 1, 0), k > 0);
                mma_commit(smem_u32(&mbar));
            }
            __syncwarp();
        }
        mbar_wait(smem_u32(&mbar), mph);
        mph ^= 1;
        tc_fence_after();
        const int row = 32 * quad + lane;
        uint32_t x[32];
        if (vb == 0) {
            tmem_ld<32>(tl, x);
            tmem_wait_ld();
            if (row < DK) {
                uint8_t* w = smem + FA_K + (row >> 6) * FA_PANEL;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    *reinterpret_cast<__nv_bfloat16*>(w + sw_off(64, 32 * half + e, row & 63)) = __float2bfloat16_rn(-__uint_as_float(x[e]));
            }
            fence_async_smem();
        }
        if (tid == 0 && vb + 1 < vblocks) load_v(vb + 1);
        tmem_ld<32>(tl + 64, x);
        tmem_wait_ld();
        if (row < int(u_cols(a.Dv))) {
            float4* u = reinterpret_cast<float4*>(fac + factor_u(DK) + vb * u_bytes(a.Dv)) + row;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
                u[(8 * half + e / 4) * int(u_cols(a.Dv))] = make_float4(__uint_as_float(x[e]), __uint_as_float(x[e + 1]),
                                                                    __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (vb == 0 && warp == 0) {
            if (elect()) {
                for (int p = 0; p < NP; ++p) bulk_store(fac + (1 + p) * T8, smem_u32(smem + FA_K + p * FA_PANEL), T8);
                bulk_commit();
                bulk_wait_read();  // shared memory is read before the CTA ends
            }
            __syncwarp();
        }
    }
    if (warp == 0) tmem_dealloc(tmem, 128);
}

// ---------------------------------------------------------------------------
// The walk over a sequence's chunks.
//
// A chunk takes 2640 cycles, 1.35 us: 128 chunks of 16 heads of 128 x 128 173 us, and the ragged
// prompts above 181 us (1.0 GB, 5.6 TB/s), where its copies and the chain are about even.  The chain is four
// hops between the products and the four groups of warps, which take a quarter of the state's rows
// and of the tokens each; the products that do not carry it (Q S, P D) are issued by a warp of their
// own in its pauses, and U = T V is formed ahead by the factors (236 to 173 us for both).
// ---------------------------------------------------------------------------
constexpr int kGroups = 4;                            // chain groups of four warps
constexpr int kWalkThreads = (4 * kGroups + 7) * 32;  // and four output warps, two of products, the copies'
constexpr int kGateRing = 8;

template <int DK>
struct WalkSmem {
    static constexpr int NP = DK / 64;
    // two of each piece: U, W, K, Q, P; then the outputs' staging and the gates
    static constexpr uint32_t U = 0, u = 4 * T8, W = U + 2 * u, w = NP * T8, K = W + 2 * w, k = NP * T8, Q = K + 2 * k,
                              q = NP * T8, P = Q + 2 * q, OUT = P + 2 * T8, GATES = OUT + 2 * T8;
    static constexpr size_t bytes = GATES + kGateRing * kGateBytes + 1024;
};
static_assert(WalkSmem<128>::bytes <= 227 * 1024, "shared memory of a CTA");

// Tensor-memory columns: A operands (bf16 pairs), then fp32 accumulators: D, the state, O twice.
constexpr uint32_t TM_S = 0, TM_DTH = 64, TM_DTL = 96, TM_DH = 128, TM_DL = 160, TM_D = 192, TM_X = 256, TM_O = 384;

// A converged warp's bounded wait; after one that ran out its others give up soon.  Every lane waits:
// try_wait then suspends the warp until the phase ends (some 60 cycles from the arrival to the next
// instruction), while a single lane's polls come back at once, take 200 to 350 cycles to notice and
// slow the products down.  The clock is read once in 64 polls.
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, bool& dead) {
    const uint32_t b = smem_u32(bar);
    uint64_t t0 = 0;
    for (uint32_t i = 1; !mbar_try_wait(b, parity); ++i) {
        if ((i & 63u) != 0) continue;
        const uint64_t t = global_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > (dead ? 1000ull * 1000 : kWaitLimitNs)) {
            atomicExch(&g_timeout_flag, 1);
            dead = true;
            break;
        }
    }
    __syncwarp();
}
// One arrival of a warp after its tensor-memory or shared-memory work.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bar));
}

struct WalkBars {
    uint64_t u_full[2], u_free[2], wkq_full[2], w_free[2], k_free[2], q_free[2], p_full[2], p_free[2];
    uint64_t gates[kGateRing];
    uint64_t s_ready[2], x_done[2], o_done[2], o_free[2], dt_ready, d_ready, d_done, fixed;
};

// How a launch of the walk divides the sequences.
//   whole   a CTA per sequence
//   first   blockIdx.z = 0: the first segment; z = j > 0: inner segment j, its dS and (one more
//           block of columns) its M
//   rest    blockIdx.z = j: segment j + 1, from the state that segment j ends with
enum class Part { whole, first, rest };
struct Segments {
    int chunks;      // of a segment
    int most;        // segments of the longest sequence
    float* ends;     // [S][H][most][Dk][Dv]: states at the segments' ends (dS before they are composed)
    float* maps;     // [S][H][most][Dk][Dk]: M
};
__device__ __forceinline__ float* end_of(const Args& a, const Segments& g, int seq, int h, int j) {
    return g.ends + ((int64_t(seq) * a.H + h) * g.most + j) * a.Dk * a.Dv;
}
__device__ __forceinline__ float* map_of(const Args& a, const Segments& g, int seq, int h, int j) {
    return g.maps + ((int64_t(seq) * a.H + h) * g.most + j) * a.Dk * a.Dk;
}

template <int DK, typename TS, Part kPart>
__global__ void __launch_bounds__(kWalkThreads, 1)
    gds_walk_kernel(const __grid_constant__ Args a, const Segments seg, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mo) {
    constexpr int NP = DK / 64;
    constexpr int GC = DK / kGroups;       // state rows (columns of tensor memory) of a group
    constexpr int GT = kChunk / kGroups;   // tokens of a group
    using L = WalkSmem<DK>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    __shared__ __align__(8) WalkBars bar;
    __shared__ uint32_t tmem_slot;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int vblocks = (a.Dv + 127) / 128, blocks = vblocks + (kPart == Part::first ? 1 : 0);
    const int h = blockIdx.x / blocks, vb = blockIdx.x % blocks;
    const bool map = vb == vblocks;  // the columns are those of M
    const int v0 = map ? 0 : vb * 128, nv = map ? DK : min(a.Dv - v0, 128);
    const int si = kPart == Part::whole ? by_length(a, blockIdx.y) : int(blockIdx.y);
    const Seq sq = sequence(a, si);
    const int all = (sq.len + kChunk - 1) / kChunk;  // the sequence's chunks
    // this CTA's segment and its chunks
    const int j = kPart == Part::whole ? 0 : int(blockIdx.z) + (kPart == Part::rest ? 1 : 0);
    const int c_first = kPart == Part::whole ? 0 : j * seg.chunks;
    // it is the sequence's last (the last one that there is takes what a sequence has beyond max_len)
    const bool ends = kPart == Part::whole || j == seg.most - 1 || c_first + seg.chunks >= all;
    const int chunks = (ends ? all : c_first + seg.chunks) - c_first;
    if (kPart != Part::whole) {
        if (j > 0 && (sq.slot < 0 || chunks <= 0)) return;
        if (kPart == Part::first && ((j > 0 && ends) || (j == 0 && map))) return;
    }
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
    const int last = ends ? sq.len - (all - 1) * kChunk : kChunk;  // tokens of the last chunk
    const bool ragged = last < kChunk;
    const int quads = (nv + 31) / 32;  // quadrants of tensor-memory lanes with columns

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            for (uint64_t* b : {&bar.u_full[i], &bar.w_free[i], &bar.k_free[i], &bar.q_free[i], &bar.p_full[i],
                                &bar.p_free[i], &bar.o_done[i]})
                mbar_init(smem_u32(b), 1);
            mbar_init(smem_u32(&bar.x_done[i]), outs ? 2 : 1);  // the state's update, and Q S, which reads the old one
            mbar_init(smem_u32(&bar.wkq_full[i]), outs ? 3 : 2);
            mbar_init(smem_u32(&bar.u_free[i]), quads * kGroups);
            mbar_init(smem_u32(&bar.s_ready[i]), quads * kGroups / 2);
            mbar_init(smem_u32(&bar.o_free[i]), quads);
        }
        for (int i = 0; i < kGateRing; ++i) mbar_init(smem_u32(&bar.gates[i]), 1);
        mbar_init(smem_u32(&bar.dt_ready), quads * kGroups);
        mbar_init(smem_u32(&bar.d_ready), quads * kGroups);
        mbar_init(smem_u32(&bar.d_done), outs ? 2 : 1);  // W S, and P D of the chunks before, whose D~ is overwritten
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

    if (warp < 4 * kGroups + 4 && ((warp & 3) >= quads || (!outs && warp >= 4 * kGroups))) {
        // no columns, or no outputs
    } else if (warp < 4 * kGroups) {
        // ---- the chain: a lane is a value column, a group a quarter of the state's rows and of the tokens
        const int grp = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);
        const bool live = row < nv;
        const int r0 = grp * GC;  // the first of this thread's rows
#pragma unroll
        for (int i0 = 0; i0 < GC; i0 += 16) {
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = r0 + i0 + i;
                float y = 0.f;
                if (kPart == Part::whole || (kPart == Part::first && j == 0)) {
                    if (live && !sq.fresh) y = to_f32(st[int64_t(r) * a.Dv + row]);
                } else if (kPart == Part::first) {
                    y = map && r == row ? 1.f : 0.f;
                } else if (live) {
                    y = end_of(a, seg, si, h, j - 1)[int64_t(r) * a.Dv + v0 + row];
                }
                x[i] = __float_as_uint(y);
            }
            tmem_st<16>(tl + TM_X + r0 + i0, x);
        }
        tmem_wait_st();
        for (int c = 0; c < chunks; ++c) {
            if (c == chunks - 1 && ragged) {
                // keys past the sequence's end are other tokens': they must not meet a zero of D~ as NaN
                wait(&bar.wkq_full[c & 1], (c >> 1) & 1, dead);
                const int at = (grp * quads + (warp & 3)) * 32 + lane;
                zero_rows(smem + L::K + (c & 1) * L::k, NP, last, at, 32 * quads * kGroups);
                fence_async_smem();
                warp_arrive(&bar.fixed, lane);
            }
            const float* gates = gates_of(c);
            const bool weak = gates[kWeak] != 0.f;
            const uint64_t end = pair(gates[kEnd], gates[kEnd]);
            if (c > 0) {
                wait(&bar.x_done[2 * grp / kGroups], (c - 1) & 1, dead);
                tc_fence_after();
            }
            {  // S~ = e^{b_63} S, to accumulate on; and S~ (or S) rounded, as an operand
                uint32_t x[GC];
                tmem_ld<GC>(tl + TM_X + grp * GC, x);
                tmem_wait_ld();
                uint32_t p[GC / 2];
                if (!weak) {
#pragma unroll
                    for (int i = 0; i < GC / 2; ++i) p[i] = pack2(pair(x[2 * i], x[2 * i + 1]));
                }
#pragma unroll
                for (int i = 0; i < GC / 2; ++i) unpair(mul2(pair(x[2 * i], x[2 * i + 1]), end), x[2 * i], x[2 * i + 1]);
                if (weak) {
#pragma unroll
                    for (int i = 0; i < GC / 2; ++i) p[i] = pack2(pair(x[2 * i], x[2 * i + 1]));
                }
                tmem_st<GC / 2>(tl + TM_S + grp * (GC / 2), p);
                tmem_st<GC>(tl + TM_X + grp * GC, x);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&bar.s_ready[2 * grp / kGroups], lane);
            }
            if (!map) wait(&bar.u_full[c & 1], (c >> 1) & 1, dead);
            ulonglong2 u[GT / 4];
#pragma unroll
            for (int i = 0; i < GT / 4; ++i)
                u[i] = map ? make_ulonglong2(0, 0)
                           : (reinterpret_cast<const ulonglong2*>(smem + L::U + (c & 1) * L::u))[(GT / 4 * grp + i) * int(u_cols(a.Dv)) + row];
            wait(&bar.d_done, c & 1, dead);
            tc_fence_after();
            uint32_t x[GT], hi[GT / 2], lo[GT / 2];
            tmem_ld<GT>(tl + TM_D + GT * grp, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < GT; i += 4) {
                unpair(add2(pair(x[i], x[i + 1]), u[i / 4].x), x[i], x[i + 1]);
                unpair(add2(pair(x[i + 2], x[i + 3]), u[i / 4].y), x[i + 2], x[i + 3]);
            }
            if (!weak) {  // D~ from D
#pragma unroll
                for (int i = 0; i < GT; i += 4) {
                    const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(gates + kDec + GT * grp + i);
                    split2(mul2(pair(x[i], x[i + 1]), e.x), hi[i / 2], lo[i / 2]);
                    split2(mul2(pair(x[i + 2], x[i + 3]), e.y), hi[i / 2 + 1], lo[i / 2 + 1]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < GT / 2; ++i) split2(pair(x[2 * i], x[2 * i + 1]), hi[i], lo[i]);
            }
            // two buffers, since P D~ of a chunk is formed in the next chunk's pauses; a chunk of strong
            // decay takes both
            const uint32_t dt = tl + (weak && (c & 1) ? TM_DH : TM_DTH) + GT / 2 * grp;
            tmem_st<GT / 2>(dt, hi);
            tmem_st<GT / 2>(dt + TM_DTL - TM_DTH, lo);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&bar.dt_ready));
                mbar_arrive(smem_u32(&bar.u_free[c & 1]));
            }
            if (!weak && outs) {  // and D itself, for P D
#pragma unroll
                for (int i = 0; i < GT / 2; ++i) split2(pair(x[2 * i], x[2 * i + 1]), hi[i], lo[i]);
                tmem_st<GT / 2>(tl + TM_DH + GT / 2 * grp, hi);
                tmem_st<GT / 2>(tl + TM_DL + GT / 2 * grp, lo);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&bar.d_ready, lane);
            }
        }
        wait(&bar.x_done[2 * grp / kGroups], (chunks - 1) & 1, dead);
        tc_fence_after();
        uint32_t x[GC];
        tmem_ld<GC>(tl + TM_X + grp * GC, x);
        tmem_wait_ld();
        if (live && ends) {
#pragma unroll
            for (int i = 0; i < GC; ++i) st[int64_t(r0 + i) * a.Dv + row] = from_f32<TS>(__uint_as_float(x[i]));
        } else if (live && kPart == Part::first) {
            float* to = map ? map_of(a, seg, si, h, j) + row : end_of(a, seg, si, h, j) + v0 + row;
#pragma unroll
            for (int i = 0; i < GC; ++i) to[int64_t(r0 + i) * (map ? DK : a.Dv)] = __uint_as_float(x[i]);
        }
        tc_fence_before();
    } else if (warp < 4 * kGroups + 4) {
        // ---- the outputs: a lane is a value column; whole chunks leave as tiles, the last one by rows
        const int w = warp & 3, row = 32 * w + lane;
        const uint32_t tl = tmem + (uint32_t(32 * w) << 16) + TM_O;
        uint8_t* tile = smem + L::OUT;
        for (int c = 0; c < chunks; ++c) {
            const float* gates = gates_of(c);
            const bool weak = gates[kWeak] != 0.f;
            const int b = c & 1;
            wait(&bar.o_done[b], (c >> 1) & 1, dead);
            tc_fence_after();
            uint32_t y[kChunk / 2];
#pragma unroll
            for (int j = 0; j < kChunk; j += 32) {
                uint32_t p[32];
                tmem_ld<32>(tl + 64 * b + j, p);
                tmem_wait_ld();
                if (weak) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(gates + j + i);
                        y[(j + i) / 2] = pack2(mul2(f.x, pair(p[i], p[i + 1])));
                        y[(j + i) / 2 + 1] = pack2(mul2(f.y, pair(p[i + 2], p[i + 3])));
                    }
                } else {  // e^b o (Q S) in this chunk's accumulator, P D in the other one
#pragma unroll
                    for (int i0 = 0; i0 < 32; i0 += 16) {
                        uint32_t q[16];
                        tmem_ld<16>(tl + 64 * (b ^ 1) + j + i0, q);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float u = fmaf(gates[j + i0 + i], __uint_as_float(p[i0 + i]), a.scale * __uint_as_float(q[i]));
                            const float v = fmaf(gates[j + i0 + i + 1], __uint_as_float(p[i0 + i + 1]), a.scale * __uint_as_float(q[i + 1]));
                            y[(j + i0 + i) / 2] = pack2(u, v);
                        }
                    }
                }
            }
            tc_fence_before();
            warp_arrive(&bar.o_free[b], lane);  // the accumulators and the decays have been read
            // the store of the chunk before has read the staging
            if (warp == 4 * kGroups && lane == 0) bulk_wait_read();
            asm volatile("bar.sync 1, %0;" ::"r"(32 * quads) : "memory");
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
                *reinterpret_cast<uint16_t*>(tile + (row >> 6) * T8 + sw_off(64, i, row & 63)) =
                    uint16_t(i & 1 ? y[i / 2] >> 16 : y[i / 2] & 0xffffu);
            const bool whole = c < chunks - 1 || !ragged;
            if (whole) fence_async_smem();
            asm volatile("bar.sync 1, %0;" ::"r"(32 * quads) : "memory");
            if (whole) {
                if (warp == 4 * kGroups && lane == 0) {
                    for (int p = 0; p < (nv + 63) / 64; ++p)
                        tma_store_3d(&mo, smem_u32(tile + p * T8), v0 + 64 * p, h, sq.begin + (c_first + c) * kChunk);
                    bulk_commit();
                }
            } else {
                for (int i = (warp & 3) * 32 + lane; i < last * 16; i += 32 * quads) {
                    const int t = i >> 4, e = (i & 15) * 8;
                    if (e < nv)
                        *reinterpret_cast<uint4*>(o + (int64_t(c) * kChunk + t) * os + e) =
                            *reinterpret_cast<const uint4*>(tile + sw_chunk(64, t, e >> 3));
                }
            }
        }
        if (warp == 4 * kGroups && lane == 0) bulk_wait_read();  // shared memory is read before the CTA ends
    } else if (warp == 4 * kGroups + 4) {
        // ---- the products of the chain.  The whole warp walks the loop and one elected lane issues, so
        // that descriptors stay in uniform registers: 30 cycles a product of N = 64 instead of 45 to 80
        // from inside a one-lane branch (measured with 8 to 64 in a row).
        const uint32_t base = smem_u32(smem);
        constexpr uint32_t kTS = idesc_bf16(128, 64, 0, 0), kTX = idesc_bf16(128, DK / 2, 0, 1);
        for (int c = 0; c < chunks; ++c) {
            const int i = c & 1;
            const uint64_t dw = sdesc(base + L::W + i * L::w, 16, 1024), dk = sdesc(base + L::K + i * L::k, T8, 1024);
            const bool weak = gates_of(c)[kWeak] != 0.f;
            wait(&bar.wkq_full[i], (c >> 1) & 1, dead);
#pragma unroll
            for (int g = 0; g < 2; ++g) {  // D^T = -S^T W^T, half of the state's rows as they come
                wait(&bar.s_ready[g], c & 1, dead);
                tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int k = g * (DK / 32); k < (g + 1) * (DK / 32); ++k)
                        mma_ts(tmem + TM_D, tmem + TM_S + 8 * k, desc_plus(dw, (k >> 2) * T8 + (k & 3) * 32), kTS, k > 0);
                    if (g == 1) {
                        mma_commit(smem_u32(&bar.d_done));
                        mma_commit(smem_u32(&bar.w_free[i]));
                    }
                }
                __syncwarp();
            }
            wait(&bar.dt_ready, c & 1, dead);
            if (c == chunks - 1 && ragged) wait(&bar.fixed, 0, dead);
            tc_fence_after();
            if (elect()) {
                const uint32_t d = tmem + (weak && i ? TM_DH : TM_DTH);
#pragma unroll
                for (int g = 0; g < 2; ++g) {  // S^T += D~^T K, half of the columns at a time
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ts(tmem + TM_X + g * (DK / 2), d + (k < 4 ? 0u : TM_DTL - TM_DTH) + 8 * (k & 3),
                               desc_plus(dk, (DK == 128 ? g * T8 : g * 64) + (k & 3) * 2048), kTX, 1);
                    if (g == 1) mma_commit(smem_u32(&bar.k_free[i]));
                    mma_commit(smem_u32(&bar.x_done[g]));
                }
            }
            __syncwarp();
        }
        for (int g = 0; g < 2; ++g) wait(&bar.x_done[g], (chunks - 1) & 1, dead);
    } else if (warp == 4 * kGroups + 5 && !outs) {
        // nothing beside the chain
    } else if (warp == 4 * kGroups + 5) {
        // ---- the products beside the chain, while it reads D: P D~ of the chunk before, then Q S
        const uint32_t base = smem_u32(smem);
        constexpr uint32_t kTS = idesc_bf16(128, 64, 0, 0);
        // O^T += D~^T P^T of chunk c (or D^T P^T on its own); an elected lane issues it
        auto pd = [&](int c, bool weak) {
            const int i = c & 1;
            const uint64_t dp = sdesc(base + L::P + i * T8, 16, 1024);
            const uint32_t d = tmem + (weak && !i ? TM_DTH : TM_DH), to = tmem + TM_O + 64 * (weak ? i : i ^ 1);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                mma_ts(to, d + (k < 4 ? 0u : TM_DTL - TM_DTH) + 8 * (k & 3), desc_plus(dp, (k & 3) * 32), kTS, weak || k > 0);
            mma_commit(smem_u32(&bar.p_free[i]));
            mma_commit(smem_u32(&bar.o_done[i]));
        };
        uint32_t strong = 0;  // chunks of strong decay so far
        bool weak = gates_of(0)[kWeak] != 0.f, was_weak = true, pending = false;
        if (elect()) mma_commit(smem_u32(&bar.d_done));
        __syncwarp();
        for (int c = 0; c < chunks; ++c) {
            const int i = c & 1;
            const uint64_t dq = sdesc(base + L::Q + i * L::q, 16, 1024);
            // every wait that does not hang on the chain is taken ahead of it.  O has two accumulators,
            // taken in turn; a chunk of strong decay takes both
            wait(&bar.wkq_full[i], (c >> 1) & 1, dead);
            if (c > 1) wait(&bar.o_free[i], ((c - 2) >> 1) & 1, dead);
            if (c > 0 && !(weak && was_weak)) wait(&bar.o_free[i ^ 1], ((c - 1) >> 1) & 1, dead);
            wait(&bar.d_done, c & 1, dead);
            tc_fence_after();
            if (elect()) {
                if (pending) pd(c - 1, true);
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)  // O^T = S^T Q^T
                    mma_ts(tmem + TM_O + 64 * i, tmem + TM_S + 8 * k, desc_plus(dq, (k >> 2) * T8 + (k & 3) * 32), kTS, k > 0);
                mma_commit(smem_u32(&bar.q_free[i]));
                mma_commit(smem_u32(&bar.x_done[0]));
                mma_commit(smem_u32(&bar.x_done[1]));
            }
            __syncwarp();
            wait(&bar.p_full[i], (c >> 1) & 1, dead);
            pending = weak;
            was_weak = weak;
            const bool more = c + 1 < chunks;
            if (more) weak = gates_of(c + 1)[kWeak] != 0.f;
            // not left for the next chunk: a chunk of strong decay, the last one, and one before a chunk of
            // strong decay, which overwrites both D~
            if (!was_weak) {
                wait(&bar.d_ready, strong & 1, dead);
                ++strong;
            } else if (!more || !weak) {
                wait(&bar.dt_ready, c & 1, dead);
            }
            tc_fence_after();
            if (elect()) {
                if (!was_weak || !more || !weak) pd(c, was_weak);
                if (more) mma_commit(smem_u32(&bar.d_done));
            }
            __syncwarp();
            if (!was_weak || !more || !weak) pending = false;
        }
        wait(&bar.o_done[(chunks - 1) & 1], ((chunks - 1) >> 1) & 1, dead);
    } else {
        // ---- the copies: each piece of chunk c once the products that read chunk c - 2's are done
        const uint32_t base = smem_u32(smem), ub = u_bytes(a.Dv), uat = factor_u(DK) + (v0 / 128) * ub;
        const uint8_t* fac = static_cast<const uint8_t*>(a.ws) + (int64_t(first_chunk(a, si) + c_first) * a.H + h) * factor_bytes(DK, a.Dv);
        for (int c = 0; c < chunks; ++c, fac += int64_t(a.H) * factor_bytes(DK, a.Dv)) {
            const int i = c & 1, ph = ((c >> 1) & 1) ^ 1, tok = sq.begin + (c_first + c) * kChunk;
            wait(&bar.u_free[i], ph, dead);
            if (elect()) {
                const uint32_t b = smem_u32(&bar.u_full[i]);
                if (!map) {
                    mbar_expect_tx(b, ub);
                    bulk_load(base + L::U + i * L::u, fac + uat, ub, b);
                }
                // the gates of chunk c - 8 are read: the products have waited for the outputs of chunk c - 5
                const uint32_t g = smem_u32(&bar.gates[c % kGateRing]);
                mbar_expect_tx(g, kGateBytes);
                bulk_load(base + L::GATES + (c % kGateRing) * kGateBytes, fac + factor_gates(DK), kGateBytes, g);
            }
            __syncwarp();
            const uint32_t b = smem_u32(&bar.wkq_full[i]);
            wait(&bar.w_free[i], ph, dead);
            if (elect()) {
                mbar_expect_tx(b, NP * T8);
                bulk_load(base + L::W + i * L::w, fac + T8, NP * T8, b);
            }
            __syncwarp();
            if (outs) {
                wait(&bar.q_free[i], ph, dead);
                if (elect()) {
                    mbar_expect_tx(b, NP * T8);
                    for (int p = 0; p < NP; ++p) tma_load_3d(base + L::Q + i * L::q + p * T8, &mq, 64 * p, h / a.hdiv, tok, b);
                }
                __syncwarp();
            }
            wait(&bar.k_free[i], ph, dead);
            if (elect()) {
                mbar_expect_tx(b, NP * T8);
                for (int p = 0; p < NP; ++p) tma_load_3d(base + L::K + i * L::k + p * T8, &mk, 64 * p, h / a.hdiv, tok, b);
            }
            __syncwarp();
            if (outs) {
                wait(&bar.p_free[i], ph, dead);
                if (elect()) {
                    const uint32_t pb = smem_u32(&bar.p_full[i]);
                    mbar_expect_tx(pb, T8);
                    bulk_load(base + L::P + i * T8, fac, T8, pb);
                }
                __syncwarp();
            }
        }
        // no copy outlives the CTA
        for (int c = max(chunks - 2, 0); c < chunks; ++c) {
            const int i = c & 1, ph = (c >> 1) & 1;
            if (!map) wait(&bar.u_full[i], ph, dead);
            wait(&bar.wkq_full[i], ph, dead);
            if (outs) wait(&bar.p_full[i], ph, dead);
            gates_of(c);
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// The states at the segments' ends, in order: E_j = M_j E_{j-1} + dS_j, E_0 from the first segment.
// A CTA takes 16 columns of a (sequence, head), a thread two columns and every 32nd row; the next M_j
// waits in registers while this one, in shared memory, is worked on (both copied into shared memory
// by bulk copies: 28 us instead of 20 for six segments of 16 heads of 128 x 128).  fp32 throughout.
constexpr int kComposeCols = 16;
template <int DK>
struct ComposeSmem {
    static constexpr uint32_t pitch = DK * 4 + 16, map = DK * pitch;  // rows in different banks
    static constexpr uint32_t E = map;
    static constexpr size_t bytes = E + DK * kComposeCols * 4 + 128;
};
template <int DK>
__global__ void __launch_bounds__(256) gds_compose_kernel(const __grid_constant__ Args a, const Segments seg) {
    constexpr int R = DK / 32;  // rows of a thread
    using L = ComposeSmem<DK>;
    extern __shared__ __align__(128) uint8_t compose_smem[];
    float2* E = reinterpret_cast<float2*>(compose_smem + L::E);  // [Dk][8] pairs of columns
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = (a.Dv + kComposeCols - 1) / kComposeCols;
    const int h = blockIdx.x / blocks, v0 = (blockIdx.x % blocks) * kComposeCols;
    const Seq sq = sequence(a, blockIdx.y);
    const int segs = min(((sq.len + kChunk - 1) / kChunk + seg.chunks - 1) / seg.chunks, seg.most);
    if (sq.slot < 0 || segs < 3) return;
    constexpr int N = DK * DK / 4 / 256;  // 16-byte units of M a thread
    float4 m4[N];
    auto fetch = [&](int j) {
        const float4* M = reinterpret_cast<const float4*>(map_of(a, seg, blockIdx.y, h, j)) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < N; ++i) m4[i] = M[i * 256];
    };
    fetch(1);
    const int c = lane & 7, r0 = 4 * warp + (lane >> 3);
    const bool live = v0 + 2 * c < a.Dv;  // (Dv is a multiple of 8)
    auto load = [&](int j, float2* x) {
        const float* end = end_of(a, seg, blockIdx.y, h, j) + v0 + 2 * c;
#pragma unroll
        for (int i = 0; i < R; ++i)
            x[i] = live ? *reinterpret_cast<const float2*>(end + int64_t(r0 + 32 * i) * a.Dv) : make_float2(0.f, 0.f);
    };
    float2 x[R], ahead[R];
    load(0, x);
    load(1, ahead);
#pragma unroll
    for (int i = 0; i < R; ++i) E[(r0 + 32 * i) * 8 + c] = x[i];
    for (int j = 1; j + 1 < segs; ++j) {
        float* end = end_of(a, seg, blockIdx.y, h, j) + v0 + 2 * c;
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = ahead[i];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = threadIdx.x + i * 256;
            *reinterpret_cast<float4*>(compose_smem + at / (DK / 4) * L::pitch + at % (DK / 4) * 16) = m4[i];
        }
        if (j + 2 < segs) {
            load(j + 1, ahead);
            fetch(j + 1);
        }
        __syncthreads();  // M and E are in place
        const uint8_t* M = compose_smem;
#pragma unroll 8
        for (int k = 0; k < DK; k += 4) {
            const float2 e0 = E[k * 8 + c], e1 = E[(k + 1) * 8 + c], e2 = E[(k + 2) * 8 + c], e3 = E[(k + 3) * 8 + c];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float4 m = *reinterpret_cast<const float4*>(M + (r0 + 32 * i) * L::pitch + k * 4);
                x[i].x = fmaf(m.w, e3.x, fmaf(m.z, e2.x, fmaf(m.y, e1.x, fmaf(m.x, e0.x, x[i].x))));
                x[i].y = fmaf(m.w, e3.y, fmaf(m.z, e2.y, fmaf(m.y, e1.y, fmaf(m.x, e0.y, x[i].y))));
            }
        }
        __syncthreads();  // and have been read
#pragma unroll
        for (int i = 0; i < R; ++i) {
            E[(r0 + 32 * i) * 8 + c] = x[i];
            if (live) *reinterpret_cast<float2*>(end + int64_t(r0 + 32 * i) * a.Dv) = x[i];
        }
    }
}

__global__ void read_flag_kernel(int* out, int clear) {
    *out = g_timeout_flag;
    if (clear) g_timeout_flag = 0;
}

// [N tokens][heads][D] bf16 with the given token and head strides; boxes of 64 tokens x 64 columns.
bool map_of(CUtensorMap* m, const void* base, int D, int heads, int N, const int64_t* strides) {
    // a dimension of one element may have any stride; the encoder wants a positive multiple of 16 bytes
    const int64_t hs = heads > 1 && strides[1] > 0 ? strides[1] : D, ts = N > 1 && strides[0] > 0 ? strides[0] : int64_t(heads) * D;
    return make_map_strided(m, base, D, heads, N, hs, ts);
}

rm_status fail(const char* what, bool map) {
    char msg[256];
    if (map) std::snprintf(msg, sizeof(msg), "gated delta rule with a carried state: no tensor map for %s (CUresult %d)", what, last_map_result());
    else std::snprintf(msg, sizeof(msg), "gated delta rule with a carried state: %s failed: %s", what, cuda_error_text());
    return api_fail(RM_ERR_CUDA, msg);
}

size_t factors_bytes(const Args& a) { return size_t(chunk_slots(a)) * a.H * factor_bytes(a.Dk, a.Dv); }

// Segments of the longest sequence (1: not cut), and their chunks.  As many as keep the first walk's
// CTAs (one per block of columns for the first segment, one more for M in each inner one) on the
// GPU's 152 multiprocessors at once, of eight chunks or more.  With n segments the chain is two walks
// of 1 / n of the chunks, some 1.2 us a chunk; two more launches and the composition cost some 30 us.  So
// a cut has to save 28 chunks.  us in a CUDA graph, whole / cut:
//     chunks                          16          32          64          128
//     16 heads of 128 x 128           38 / 54     68 / 76     122 / 111   230 / 176 (strong decay 232 / 176)
//     two prompts of 8 such heads                 68 / 79                 230 / 176
//     32 heads of 128 x 128                       82 / 102                278 / 277
//     48 heads of 128 x 128                                               331 / 360
//     16 heads of 64 x 64                         55 / 55                 185 / 128
//     4 heads of 64 x 64                                      81 / 51
//     8 heads of 128 x 256                        61 / 65                 211 / 150
//     16 heads of 128 x 256 (4 segments)                                  242 / 226
// and with three segments the second walk shares the memory with too many others to gain.
int segments(const Args& a, int* chunks) {
    const int all = (a.max_len + kChunk - 1) / kChunk, blocks = (a.Dv + 127) / 128;
    const int each = 152 / (a.H * a.S);  // CTAs of a sequence's head
    int n = each > blocks ? 2 + (each - blocks) / (blocks + 1) : 1;
    n = n < kMostSegments ? n : kMostSegments;
    n = n < all / 8 ? n : all / 8;
    if (n < 4 || all * (n - 2) < 28 * n) return 1;
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
    auto ff = gds_factor_kernel<DK>;
    if (!set_smem(ff, kFactorSmem)) return fail("shared-memory attribute of the factors", false);
    ff<<<dim3(unsigned(chunk_slots(a)), unsigned(a.H)), 256, kFactorSmem, s>>>(a, mq, mk, mv);
    note_launch(1);
    if (!launch_ok()) return fail("launch of the factors", false);
    Segments seg{0, 1, nullptr, nullptr};
    const int segs = segments(a, &seg.chunks);
    const unsigned blocks = unsigned((a.Dv + 127) / 128);
    auto walk = [&](auto f, dim3 grid) {
        if (!set_smem(f, WalkSmem<DK>::bytes)) return fail("shared-memory attribute of the walk", false);
        f<<<grid, kWalkThreads, WalkSmem<DK>::bytes, s>>>(a, seg, mq, mk, mo);
        note_launch(1);
        return launch_ok() ? RM_OK : fail("launch of the walk", false);
    };
    const bool f = state_dt == RM_F32;
    if (segs == 1)
        return f ? walk(gds_walk_kernel<DK, float, Part::whole>, dim3(blocks * a.H, a.S))
                 : walk(gds_walk_kernel<DK, __nv_bfloat16, Part::whole>, dim3(blocks * a.H, a.S));
    seg.most = segs;
    seg.ends = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + factors_bytes(a));
    seg.maps = seg.ends + int64_t(a.S) * a.H * segs * a.Dk * a.Dv;
    const dim3 g1((blocks + 1) * a.H, a.S, segs - 1), g2(blocks * a.H, a.S, segs - 1);
    rm_status st = f ? walk(gds_walk_kernel<DK, float, Part::first>, g1) : walk(gds_walk_kernel<DK, __nv_bfloat16, Part::first>, g1);
    if (st != RM_OK) return st;
    auto fc = gds_compose_kernel<DK>;
    if (!set_smem(fc, ComposeSmem<DK>::bytes)) return fail("shared-memory attribute of the composition", false);
    fc<<<dim3(unsigned((a.Dv + kComposeCols - 1) / kComposeCols * a.H), unsigned(a.S)), 256, ComposeSmem<DK>::bytes, s>>>(a, seg);
    note_launch(1);
    if (!launch_ok()) return fail("launch of the composition", false);
    st = f ? walk(gds_walk_kernel<DK, float, Part::rest>, g2) : walk(gds_walk_kernel<DK, __nv_bfloat16, Part::rest>, g2);
    if (st != RM_OK) return st;
    return RM_OK;
}

}  // namespace

bool tc_supports(const Args& a, rm_dtype dt) {
    return !a.recurrent && dt == RM_BF16 && (a.Dk == 64 || a.Dk == 128) && a.max_len >= kChunkedLen && a.H <= 65535;
}

// A smaller problem may be cut into more segments than this one, so the bound is that of all of them:
// n <= 2 + (152 / (heads sequences) - 1) / 2, and four or more only for heads x sequences <= 30, so
// heads x sequences x n <= 2 x 30 + 152 / 2 = 136.
size_t tc_workspace_bytes(const Args& a) {
    return factors_bytes(a) + size_t(kMostStates) * (size_t(a.Dk) * a.Dv + size_t(a.Dk) * a.Dk) * sizeof(float);
}

rm_status tc_launch(const Args& a, rm_dtype state_dt, cudaStream_t s) {
    return a.Dk == 64 ? launch<64>(a, state_dt, s) : launch<128>(a, state_dt, s);
}

}  // namespace gds

rm_status gdstc_read_timeout_flag(int* host_flag, int clear, int* dev_scratch, cudaStream_t s) {
    gds::read_flag_kernel<<<1, 1, 0, s>>>(dev_scratch, clear);
    if (!launch_ok()) return RM_ERR_CUDA;
    note_launch(1);
    if (cudaMemcpyAsync(host_flag, dev_scratch, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return RM_ERR_CUDA;
    return cudaStreamSynchronize(s) == cudaSuccess ? RM_OK : RM_ERR_CUDA;
}

}  // namespace rmcp
