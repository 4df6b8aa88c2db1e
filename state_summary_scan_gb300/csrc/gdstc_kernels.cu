// gdstc_kernels.cu -- the gated delta rule with a carried state in chunks of 64 tokens on the
// tensor cores (tcgen05 + TMA): ragged prompts in bf16, Dk in {64, 128}, any Dv.
//
// With b_t the running sum of a chunk's gates, gam_t = e^{b_t}, Gam[t][r] = e^{b_t - b_r} (r <= t),
// A[t][r] = beta_t (k_t.k_r) Gam[t][r] (r < t), T = (I + A)^{-1} diag(beta) and S the state before
// the chunk, unrolling the recurrence gives (the WY form of the product of I - beta k k^T):
//     D  = T V - W S,               W = T (K o gam)
//     O  = scale gam o (Q S) + P D, P = scale mask(Q K^T) o Gam
//     S' = e^{b_63} S + K^T D~,     D~_t = e^{b_63 - b_t} D_t
// Two launches:
//   gds_factor_kernel  every (chunk, head) at once: T, P, -W and the decays, which do not depend
//                      on the state, as images of the swizzled tiles that the walk copies in
//   gds_walk_kernel    one CTA per (sequence, head, 128 columns of values): the chain over the
//                      sequence's chunks
//
// The walk is bound by the latency of its chain: S -> W S -> D -> K^T D~ -> S.  It keeps S
// transposed, a value column a lane, so that every step of the chain is a row of tensor memory
// per thread and the rounded S and D go back to tensor memory as A operands, with no transposition
// and no shared memory; the state itself stays in fp32 registers.  Products that do not carry the
// chain (T V of the next chunk, Q S, P D) are issued behind those that do, and the outputs are
// read and stored by warps of their own.
//
// Rounding: K, Q and V enter as they are; T, D and D~ as the sum of two bf16 (16 significant
// bits: two products with the exact operand), because T's and D's errors reach the state
// undamped.  S, W and P are rounded once to bf16: S and W only enter through W S, which is small
// beside T V, and P only through O, which is rounded to bf16 anyway.  In fp64 with these roundings alone
// (1024 tokens, 4 heads of 128): state 1.4e-4 off, o 2.4e-3 with its own rounding of 1.7e-3.
#include <cstdio>

#include "gds.cuh"
#include "gdr_tri.cuh"

namespace rmcp {
namespace gds {

using namespace tc;

namespace {

constexpr uint32_t T8 = kTileBytes;      // one [64][64] bf16 tile
constexpr uint32_t kGateBytes = 1024;    // gam [64], dec [64], e^{b_63}, padding
constexpr float kForget = -110.f;        // e^{-110} is 0 in fp32: lower gates are raised to it

// Factors of a (chunk, head) in the workspace: T hi, T lo, P, -W (Dk / 64 tiles), gates.
__host__ __device__ constexpr uint32_t factor_bytes(int Dk) { return (3 + Dk / 64) * T8 + kGateBytes; }

// First chunk of sequence i: chunks of different sequences do not meet, since a sequence of n
// tokens from token b has at most floor((b + n) / 64) - floor(b / 64) + 1 of them.
__device__ __forceinline__ int first_chunk(const Args& a, int i) {
    const int b = a.cu ? min(max(__ldg(a.cu + i), 0), a.N) : i * a.each;
    return b / kChunk + i;
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

// true in one lane of a converged warp
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n.reg .pred P;\nelect.sync _|P, 0xffffffff;\nselp.u32 %0, 1, 0, P;\n}\n" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&p);
}
// the parts of x and y that pack2(x, y) leaves
__device__ __forceinline__ uint32_t pack2_rest(float x, float y, uint32_t hi) {
    return pack2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

// Zero rows [n, 64) of `tiles` adjacent [64][64] tiles.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int tiles, int n, int tid, int threads) {
    const int each = (kChunk - n) * 8;  // 16-byte units of a tile
    for (int i = tid; i < tiles * each; i += threads)
        *reinterpret_cast<uint4*>(tile + (i / each) * T8 + n * 128 + (i % each) * 16) = make_uint4(0, 0, 0, 0);
}

// Xs = (I + La)^{-1} for the strictly lower La ([64][64] fp32, pitches kP and kQ; see gdr_tri.cuh),
// by halves: the four 16 x 16 diagonal blocks by forward substitution (a column's rows in 16
// lanes), then twice the block below the diagonal of a pair, X21 = -X22 (A21 X11).  A21 X11 waits in
// the pair's block above the diagonal, so that nothing but La and Xs is needed and three CTAs fit an
// SM; entries above the diagonal are not zero afterwards.  All 256 threads call it.
__device__ __forceinline__ void halves_inverse(const float* La, float* Xs) {
    using gdrtc::kP;
    using gdrtc::kQ;
    const int tid = threadIdx.x;
    {
        const int w = tid >> 5, lane = tid & 31;
        const int o = 16 * (w >> 1), r = lane & 15, grp = ((w & 1) << 1) | (lane >> 4);
        float x[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = r == 4 * grp + m ? 1.f : 0.f;
        const float* lrow = La + (o + r) * kP + o;
#pragma unroll
        for (int k = 0; k < 15; ++k) {
            const float l = r > k ? lrow[k] : 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m) x[m] = fmaf(-l, __shfl_sync(kFull, x[m], (lane & 16) | k), x[m]);
        }
        *reinterpret_cast<float4*>(Xs + (o + r) * kQ + o + 4 * grp) = make_float4(x[0], x[1], x[2], x[3]);
    }
    __syncthreads();
    // one product of a level: out[r][4 q ..] = f sum_k a[r][k] b[k][4 q ..], n terms
    auto product = [&](const float* arow, const float* b, float* out, int n, float f) {
        float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const float l = arow[k];
            const float4 v = *reinterpret_cast<const float4*>(b + k * kQ);
            a0 = fmaf(l, v.x, a0);
            a1 = fmaf(l, v.y, a1);
            a2 = fmaf(l, v.z, a2);
            a3 = fmaf(l, v.w, a3);
        }
        *reinterpret_cast<float4*>(out) = make_float4(f * a0, f * a1, f * a2, f * a3);
    };
    {  // pairs of 16: 64 threads each
        const int o = 32 * ((tid >> 6) & 1), r = (tid >> 2) & 15, q = 4 * (tid & 3);
        if (tid < 128) product(La + (o + 16 + r) * kP + o, Xs + o * kQ + o + q, Xs + (o + r) * kQ + o + 16 + q, 16, 1.f);
        __syncthreads();
        if (tid < 128) product(Xs + (o + 16 + r) * kQ + o + 16, Xs + o * kQ + o + 16 + q, Xs + (o + 16 + r) * kQ + o + q, 16, -1.f);
        __syncthreads();
    }
    {  // the pair of 32.  X11's block above its diagonal holds sums, not zeros: its terms of row
       // k < 16 and column 16 + c are left out (and X22's below)
        const int r = tid >> 3, q = 4 * (tid & 7);
        if (q < 16) product(La + (32 + r) * kP, Xs + q, Xs + r * kQ + 32 + q, 32, 1.f);
        else product(La + (32 + r) * kP + 16, Xs + 16 * kQ + q, Xs + r * kQ + 32 + q, 16, 1.f);
        __syncthreads();
        product(Xs + (32 + r) * kQ + 32, Xs + 32 + q, Xs + (32 + r) * kQ + q, r < 16 ? 16 : 32, -1.f);
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// The factors of every (chunk, head).  Rows past the sequence's end have beta = 0, a zero key
// and a zero row of P, so that they write nothing and read nothing.
// ---------------------------------------------------------------------------
template <int DK>
struct FactorSmem {
    // staged results lie over what they no longer need: P over Q, T (hi, lo) over A, -W over K
    static constexpr uint32_t K = 0, Q = (DK / 64) * T8, A = 2 * (DK / 64) * T8, T = A, X = A + 17 * 1024;
    static constexpr size_t bytes = X + 17 * 1024 + 1024;
    static_assert(gdrtc::kD * gdrtc::kQ * 4 <= 17 * 1024, "X");
};

template <int DK>
__global__ void __launch_bounds__(256, 3)
    gds_factor_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap mq,
                      const __grid_constant__ CUtensorMap mk) {
    constexpr int NP = DK / 64;
    using L = FactorSmem<DK>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    float* La = reinterpret_cast<float*>(smem + L::A);
    float* Xs = reinterpret_cast<float*>(smem + L::X);
    __shared__ __align__(16) float b_s[kChunk], beta_s[kChunk], gam_s[kChunk];
    __shared__ __align__(8) uint64_t full, mbar;
    __shared__ uint32_t tmem_slot;

    const Geo G = geo();
    const int c = blockIdx.x, h = blockIdx.y;
    // the sequence of this chunk slot: the last one whose first chunk is at or before it
    int lo = 0, hi = a.S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_chunk(a, mid) <= c) lo = mid;
        else hi = mid - 1;
    }
    const Seq sq = sequence(a, lo);
    const int t0 = (c - first_chunk(a, lo)) * kChunk;
    if (t0 < 0 || t0 >= sq.len || sq.slot < 0) return;
    const int n = min(sq.len - t0, kChunk);  // tokens of the chunk
    const int64_t tok = sq.begin + t0;

    if (G.tid == 0) {
        mbar_init(smem_u32(&full), 1);
        mbar_init(smem_u32(&mbar), 1);
        mbar_fence_init();
    }
    if (G.warp == 0) tmem_alloc(smem_u32(&tmem_slot), 128);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;  // [0,64) K K^T, [64,128) Q K^T; then [0,DK) W
    if (G.tid == 0) {
        mbar_expect_tx(smem_u32(&full), 2 * NP * T8);
        for (int p = 0; p < NP; ++p) {
            tma_load_3d(smem_u32(smem + L::K + p * T8), &mk, 64 * p, h / a.hdiv, int(tok), smem_u32(&full));
            tma_load_3d(smem_u32(smem + L::Q + p * T8), &mq, 64 * p, h / a.hdiv, int(tok), smem_u32(&full));
        }
    }
    if (G.warp == 0) {  // the running sum of the gates, two tokens a lane
        float g[2], be[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * G.lane + i;
            g[i] = t < n ? __ldg(a.g + (tok + t) * a.gs + h) : 0.f;
            be[i] = t < n ? __ldg(a.beta + (tok + t) * a.bs + h) : 0.f;
            g[i] = g[i] < kForget ? kForget : g[i];
        }
        float ps = g[0] + g[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(kFull, ps, o);
            if (G.lane >= o) ps += x;
        }
        const float end = __shfl_sync(kFull, ps, 31);
        const float b[2] = {ps - g[1], ps};
        float* gates = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) +
                                                (int64_t(c) * a.H + h) * factor_bytes(DK) + (3 + NP) * T8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * G.lane + i;
            b_s[t] = b[i];
            beta_s[t] = be[i];
            gam_s[t] = expf(b[i]);
            gates[t] = a.scale * expf(b[i]);
            gates[64 + t] = expf(end - b[i]);
        }
        if (G.lane == 0) gates[128] = expf(end);
    }
    mbar_wait(smem_u32(&full), 0);
    if (n < kChunk) {
        zero_rows(smem + L::K, NP, n, G.tid, 256);
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint64_t DKK = sdesc(smem_u32(smem + L::K), 16, 1024), DQ = sdesc(smem_u32(smem + L::Q), 16, 1024);
    uint32_t mph = 0;
    if (G.tid == 0) {
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) {
            const uint32_t at = (k >> 2) * T8 + (k & 3) * 32;
            mma_bf16(tmem, desc_plus(DKK, at), desc_plus(DKK, at), idesc_bf16(64, 64, 0, 0), k > 0);
            mma_bf16(tmem + 64, desc_plus(DQ, at), desc_plus(DKK, at), idesc_bf16(64, 64, 0, 0), k > 0);
        }
        mma_commit(smem_u32(&mbar));
    }
    mbar_wait(smem_u32(&mbar), mph);
    mph ^= 1;
    tc_fence_after();
    uint8_t* fac = static_cast<uint8_t*>(a.ws) + (int64_t(c) * a.H + h) * factor_bytes(DK);
    const int c0 = 32 * G.grp + 16 * G.hi;
    {
        float kk[16], qk[16], p[16];
        tok16x2(tmem, G, 32 * G.grp, 64 + 32 * G.grp, kk, qk);
        const float bt = b_s[G.tau], be = beta_s[G.tau];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int r = c0 + e;
            const float m = __expf(bt - b_s[r]);
            La[G.tau * gdrtc::kP + r] = r < G.tau ? be * kk[e] * m : 0.f;
            p[e] = r <= G.tau && G.tau < n ? a.scale * qk[e] * m : 0.f;
        }
        store_row16(smem + L::Q, G.tau, c0, p);
    }
    // K o gam over K (its products are done)
#pragma unroll
    for (int p = 0; p < NP; ++p) gdrtc::rows_scaled(smem + L::K + p * T8, smem + L::K + p * T8, gam_s, 1.f, G.tid);
    __syncthreads();
    halves_inverse(La, Xs);
    {
        float x[16], lo16[16];
        gdrtc::xs_row16(Xs, G.tau, c0, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            x[e] = c0 + e <= G.tau ? x[e] * beta_s[c0 + e] : 0.f;
            lo16[e] = x[e] - __bfloat162float(__float2bfloat16_rn(x[e]));
        }
        store_row16(smem + L::T, G.tau, c0, x);
        store_row16(smem + L::T + T8, G.tau, c0, lo16);
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (G.tid == 0) {  // W = T (K o gam): K o gam is [tokens][Dk], MN-major
        const uint64_t DT = sdesc(smem_u32(smem + L::T), 16, 1024), DM = sdesc(smem_u32(smem + L::K), T8, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mma_bf16(tmem, desc_plus(DT, k * 32), desc_plus(DM, k * 2048), idesc_bf16(64, DK, 0, 1), k > 0);
        mma_commit(smem_u32(&mbar));
        bulk_store(fac, smem_u32(smem + L::T), 2 * T8);
        bulk_store(fac + 2 * T8, smem_u32(smem + L::Q), T8);
        bulk_commit();
    }
    mbar_wait(smem_u32(&mbar), mph);
    tc_fence_after();
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        float w[16];
        tok16(tmem, G, 64 * p + 32 * G.grp, w);
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = -w[e];
        store_row16(smem + L::K + p * T8, G.tau, c0, w);
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    if (G.tid == 0) {
        bulk_store(fac + 3 * T8, smem_u32(smem + L::K), NP * T8);
        bulk_commit();
        bulk_wait_read();  // shared memory is read before the CTA ends
    }
    if (G.warp == 0) tmem_dealloc(tmem, 128);
}

// ---------------------------------------------------------------------------
// The walk over a sequence's chunks.
// ---------------------------------------------------------------------------
constexpr int kGroups = 4;                            // chain groups of four warps
constexpr int kWalkThreads = (4 * kGroups + 6) * 32;  // and four output warps, the products', the copies'
constexpr int kGateRing = 4;

template <int DK>
struct WalkSmem {
    static constexpr int NP = DK / 64;
    // two of each piece, every one with barriers of its own: V with T, W, K, Q with P
    static constexpr uint32_t VT = 0, vt = 4 * T8, W = VT + 2 * vt, w = NP * T8, K = W + 2 * w, k = NP * T8, QP = K + 2 * k,
                              qp = (NP + 1) * T8, GATES = QP + 2 * qp;
    static constexpr size_t bytes = GATES + kGateRing * kGateBytes + 1024;
};
static_assert(WalkSmem<128>::bytes <= 227 * 1024, "shared memory of a CTA");

// Tensor-memory columns: A operands (bf16 pairs), then fp32 accumulators.
constexpr uint32_t TM_S = 0, TM_DTH = 64, TM_DTL = 96, TM_DH = 128, TM_DL = 160, TM_D = 192, TM_X = 256, TM_O1 = 384,
                   TM_O2 = 448;

// A bounded wait; after one that ran out the others of this thread give up soon.
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, bool& dead) {
    if (!mbar_wait(smem_u32(bar), parity, dead ? 1000ull * 1000 : kWaitLimitNs)) dead = true;
}
// One arrival of a warp after its tensor-memory or shared-memory work.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bar));
}

struct WalkBars {
    uint64_t vt_full[2], vt_free[2], w_full[2], w_free[2], k_full[2], k_free[2], qp_full[2], qp_free[2];
    uint64_t gates[kGateRing];
    uint64_t s_ready[kGroups], x_done[2], dt_ready, d_ready, d_done, o_done, o_free, fixed;
};

template <int DK, typename TS>
__global__ void __launch_bounds__(kWalkThreads, 1)
    gds_walk_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap mq,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    constexpr int NP = DK / 64;
    constexpr int GC = DK / kGroups;       // state rows (columns of tensor memory) of a group
    constexpr int GT = kChunk / kGroups;   // tokens of a group
    using L = WalkSmem<DK>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024(smem_raw);
    __shared__ __align__(8) WalkBars bar;
    __shared__ uint32_t tmem_slot;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blocks = (a.Dv + 127) / 128;
    const int h = blockIdx.x / blocks, v0 = (blockIdx.x % blocks) * 128, nv = min(a.Dv - v0, 128);
    const Seq sq = sequence(a, blockIdx.y);
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + (int64_t(sq.begin) * a.H + h) * a.Dv + v0;
    const int64_t os = int64_t(a.H) * a.Dv;
    TS* st = static_cast<TS*>(a.state) + (int64_t(max(sq.slot, 0)) * a.H + h) * DK * a.Dv + v0;
    if (sq.slot < 0) {  // padding
        for (int i = tid; i < sq.len * (nv / 8); i += kWalkThreads)
            *reinterpret_cast<uint4*>(o + (i / (nv / 8)) * os + (i % (nv / 8)) * 8) = make_uint4(0, 0, 0, 0);
        return;
    }
    if (sq.len == 0) {
        if (sq.fresh)
            for (int i = tid; i < DK * nv; i += kWalkThreads) st[int64_t(i / nv) * a.Dv + i % nv] = from_f32<TS>(0.f);
        return;
    }
    const int chunks = (sq.len + kChunk - 1) / kChunk, last = sq.len - (chunks - 1) * kChunk;
    const bool ragged = last < kChunk;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            for (uint64_t* b : {&bar.vt_full[i], &bar.vt_free[i], &bar.w_full[i], &bar.w_free[i], &bar.k_full[i], &bar.k_free[i],
                                &bar.qp_full[i], &bar.qp_free[i], &bar.x_done[i]})
                mbar_init(smem_u32(b), 1);
        }
        for (int i = 0; i < kGateRing; ++i) mbar_init(smem_u32(&bar.gates[i]), 1);
        for (int i = 0; i < kGroups; ++i) mbar_init(smem_u32(&bar.s_ready[i]), 4);
        mbar_init(smem_u32(&bar.dt_ready), 4 * kGroups);
        mbar_init(smem_u32(&bar.d_ready), 4 * kGroups);
        mbar_init(smem_u32(&bar.d_done), 1);
        mbar_init(smem_u32(&bar.o_done), 1);
        mbar_init(smem_u32(&bar.o_free), 4);
        mbar_init(smem_u32(&bar.fixed), 4 * kGroups);
        mbar_fence_init();
    }
    if (warp == 0) tmem_alloc(smem_u32(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    bool dead = false;

    if (warp < 4 * kGroups) {
        // ---- the chain: a lane is a value column, a group a quarter of the state's rows and of the tokens
        const int grp = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);
        const bool live = row < nv;
        float S[GC];
        TS* mine = st + int64_t(grp * GC) * a.Dv + row;
#pragma unroll
        for (int i = 0; i < GC; ++i) S[i] = live && !sq.fresh ? to_f32(mine[int64_t(i) * a.Dv]) : 0.f;
        float end = 1.f;
        for (int c = 0; c <= chunks; ++c) {
            if (c == chunks - 1 && ragged) {
                // rows past the sequence's end hold other tokens: they must not meet a zero of D or T as NaN
                wait(&bar.vt_full[c & 1], (c >> 1) & 1, dead);
                wait(&bar.k_full[c & 1], (c >> 1) & 1, dead);
                zero_rows(smem + L::VT + (c & 1) * L::vt, 2, last, tid, 128 * kGroups);
                zero_rows(smem + L::K + (c & 1) * L::k, NP, last, tid, 128 * kGroups);
                fence_async_smem();
                warp_arrive(&bar.fixed, lane);
            }
            if (c > 0) {
                wait(&bar.x_done[grp >> 1], (c - 1) & 1, dead);
                tc_fence_after();
                uint32_t x[GC];
                tmem_ld<GC>(tl + TM_X + grp * GC, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < GC; ++i) S[i] = fmaf(end, S[i], __uint_as_float(x[i]));
                if (c == chunks) break;
            }
            {
                uint32_t p[GC / 2];
#pragma unroll
                for (int i = 0; i < GC / 2; ++i) p[i] = pack2(S[2 * i], S[2 * i + 1]);
                tmem_st<GC / 2>(tl + TM_S + grp * (GC / 2), p);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&bar.s_ready[grp], lane);
            }
            // the decays of this group's tokens, while the product runs
            const float* gates = reinterpret_cast<const float*>(smem + L::GATES + (c % kGateRing) * kGateBytes);
            wait(&bar.gates[c % kGateRing], (c / kGateRing) & 1, dead);
            float dec[GT];
#pragma unroll
            for (int i = 0; i < GT; i += 4) {
                const float4 e = *reinterpret_cast<const float4*>(gates + 64 + GT * grp + i);
                dec[i] = e.x, dec[i + 1] = e.y, dec[i + 2] = e.z, dec[i + 3] = e.w;
            }
            end = gates[128];
            wait(&bar.d_done, c & 1, dead);
            tc_fence_after();
            uint32_t x[GT], hi[GT / 2], lo[GT / 2];
            tmem_ld<GT>(tl + TM_D + GT * grp, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < GT / 2; ++i) {  // D~, which the chain waits for, first
                const float u = __uint_as_float(x[2 * i]) * dec[2 * i], w = __uint_as_float(x[2 * i + 1]) * dec[2 * i + 1];
                hi[i] = pack2(u, w);
                lo[i] = pack2_rest(u, w, hi[i]);
            }
            tmem_st<GT / 2>(tl + TM_DTH + GT / 2 * grp, hi);
            tmem_st<GT / 2>(tl + TM_DTL + GT / 2 * grp, lo);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&bar.dt_ready, lane);
#pragma unroll
            for (int i = 0; i < GT / 2; ++i) {
                const float u = __uint_as_float(x[2 * i]), w = __uint_as_float(x[2 * i + 1]);
                hi[i] = pack2(u, w);
                lo[i] = pack2_rest(u, w, hi[i]);
            }
            tmem_st<GT / 2>(tl + TM_DH + GT / 2 * grp, hi);
            tmem_st<GT / 2>(tl + TM_DL + GT / 2 * grp, lo);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&bar.d_ready, lane);
        }
        if (live) {
#pragma unroll
            for (int i = 0; i < GC; ++i) mine[int64_t(i) * a.Dv] = from_f32<TS>(S[i]);
        }
        tc_fence_before();
    } else if (warp < 4 * kGroups + 4) {
        // ---- the outputs: a lane is a value column, so a warp stores 64 bytes of a token at a time
        const int w = warp & 3, row = 32 * w + lane;
        const uint32_t tl = tmem + (uint32_t(32 * w) << 16);
        __nv_bfloat16* mine = o + row;
        for (int c = 0; c < chunks; ++c) {
            const float* gam = reinterpret_cast<const float*>(smem + L::GATES + (c % kGateRing) * kGateBytes);
            wait(&bar.gates[c % kGateRing], (c / kGateRing) & 1, dead);
            wait(&bar.o_done, c & 1, dead);
            tc_fence_after();
            const int n = c == chunks - 1 ? last : kChunk;
#pragma unroll
            for (int j = 0; j < kChunk; j += 16) {
                uint32_t p[16], q[16];
                tmem_ld<16>(tl + TM_O1 + j, p);
                tmem_ld<16>(tl + TM_O2 + j, q);
                tmem_wait_ld();
                float y[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = fmaf(gam[j + i], __uint_as_float(p[i]), __uint_as_float(q[i]));
                if (j == kChunk - 16) {  // the accumulators and the decays have been read
                    tc_fence_before();
                    warp_arrive(&bar.o_free, lane);
                }
                if (row < nv) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (j + i < n) mine[(j + i) * os] = __float2bfloat16_rn(y[i]);
                }
            }
            mine += kChunk * os;
        }
    } else if (warp == 4 * kGroups + 4) {
        // ---- the products.  The whole warp walks the loop and one elected lane issues, so that
        // descriptors stay in uniform registers: 30 cycles a product of N = 64 instead of 45 to 80
        // from inside a one-lane branch (measured with 8 to 64 in a row).
        const uint32_t base = smem_u32(smem);
        constexpr uint32_t kTV = idesc_bf16(128, 64, 1, 0), kTS = idesc_bf16(128, 64, 0, 0), kTX = idesc_bf16(128, DK / 2, 0, 1);
        // D^T = V^T T^T of chunk c (T as the sum of two)
        auto tv = [&](int c) {
            wait(&bar.vt_full[c & 1], (c >> 1) & 1, dead);
            if (c == chunks - 1 && ragged) wait(&bar.fixed, 0, dead);
            tc_fence_after();
            const uint32_t s = base + L::VT + (c & 1) * L::vt;
            const uint64_t dv = sdesc(s, T8, 1024), dt = sdesc(s + 2 * T8, 16, 1024);
            if (elect()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_bf16(tmem + TM_D, desc_plus(dv, (k & 3) * 2048), desc_plus(dt, (k >> 2) * T8 + (k & 3) * 32), kTV, k > 0);
                mma_commit(smem_u32(&bar.vt_free[c & 1]));
            }
            __syncwarp();
        };
        tv(0);
        for (int c = 0; c < chunks; ++c) {
            const int i = c & 1, ph = (c >> 1) & 1;
            const uint64_t dw = sdesc(base + L::W + i * L::w, 16, 1024), dk = sdesc(base + L::K + i * L::k, T8, 1024);
            const uint64_t dq = sdesc(base + L::QP + i * L::qp, 16, 1024), dp = desc_plus(dq, NP * T8);
            wait(&bar.w_full[i], ph, dead);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {  // D^T -= S^T W^T, each group's rows of the state as they come
                wait(&bar.s_ready[g], c & 1, dead);
                tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int k = g * (GC / 16); k < (g + 1) * (GC / 16); ++k)
                        mma_ts(tmem + TM_D, tmem + TM_S + 8 * k, desc_plus(dw, (k >> 2) * T8 + (k & 3) * 32), kTS, 1);
                    if (g == kGroups - 1) {
                        mma_commit(smem_u32(&bar.d_done));
                        mma_commit(smem_u32(&bar.w_free[i]));
                    }
                }
                __syncwarp();
            }
            wait(&bar.qp_full[i], ph, dead);
            if (c > 0) wait(&bar.o_free, (c - 1) & 1, dead);
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)  // O1^T = S^T Q^T
                    mma_ts(tmem + TM_O1, tmem + TM_S + 8 * k, desc_plus(dq, (k >> 2) * T8 + (k & 3) * 32), kTS, k > 0);
            }
            __syncwarp();
            wait(&bar.k_full[i], ph, dead);
            wait(&bar.dt_ready, c & 1, dead);
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {  // X^T = D~^T K, half of the columns at a time
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ts(tmem + TM_X + g * (DK / 2), tmem + (k < 4 ? TM_DTH : TM_DTL) + 8 * (k & 3),
                               desc_plus(dk, (DK == 128 ? g * T8 : g * 64) + (k & 3) * 2048), kTX, k > 0);
                    mma_commit(smem_u32(&bar.x_done[g]));
                }
                mma_commit(smem_u32(&bar.k_free[i]));
            }
            __syncwarp();
            wait(&bar.d_ready, c & 1, dead);
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)  // O2^T = D^T P^T
                    mma_ts(tmem + TM_O2, tmem + (k < 4 ? TM_DH : TM_DL) + 8 * (k & 3), desc_plus(dp, (k & 3) * 32), kTS, k > 0);
                mma_commit(smem_u32(&bar.o_done));
                mma_commit(smem_u32(&bar.qp_free[i]));
            }
            __syncwarp();
            if (c + 1 < chunks) tv(c + 1);
        }
        wait(&bar.x_done[1], (chunks - 1) & 1, dead);
        wait(&bar.o_done, (chunks - 1) & 1, dead);
    } else {
        // ---- the copies: each piece of chunk c once the products that read chunk c - 2's are done
        if (lane == 0) {
            const uint32_t vt = (nv + 63) / 64, base = smem_u32(smem);
            const uint8_t* fac = static_cast<const uint8_t*>(a.ws) + (int64_t(first_chunk(a, blockIdx.y)) * a.H + h) * factor_bytes(DK);
            for (int c = 0; c < chunks; ++c, fac += int64_t(a.H) * factor_bytes(DK)) {
                const int i = c & 1, ph = ((c >> 1) & 1) ^ 1, tok = sq.begin + c * kChunk;
                uint32_t b = smem_u32(&bar.vt_full[i]), s = base + L::VT + i * L::vt;
                wait(&bar.vt_free[i], ph, dead);
                // the gates of chunk c - 4 are read: V and T of chunk c - 2 are, which follows
                const uint32_t gb = smem_u32(&bar.gates[c % kGateRing]);
                mbar_expect_tx(gb, kGateBytes);
                bulk_load(base + L::GATES + (c % kGateRing) * kGateBytes, fac + (3 + NP) * T8, kGateBytes, gb);
                mbar_expect_tx(b, (vt + 2) * T8);
                for (uint32_t p = 0; p < vt; ++p) tma_load_3d(s + p * T8, &mv, v0 + 64 * p, h, tok, b);
                bulk_load(s + 2 * T8, fac, 2 * T8, b);
                wait(&bar.w_free[i], ph, dead);
                b = smem_u32(&bar.w_full[i]);
                mbar_expect_tx(b, NP * T8);
                bulk_load(base + L::W + i * L::w, fac + 3 * T8, NP * T8, b);
                wait(&bar.k_free[i], ph, dead);
                b = smem_u32(&bar.k_full[i]);
                mbar_expect_tx(b, NP * T8);
                for (int p = 0; p < NP; ++p) tma_load_3d(base + L::K + i * L::k + p * T8, &mk, 64 * p, h / a.hdiv, tok, b);
                wait(&bar.qp_free[i], ph, dead);
                b = smem_u32(&bar.qp_full[i]), s = base + L::QP + i * L::qp;
                mbar_expect_tx(b, (NP + 1) * T8);
                for (int p = 0; p < NP; ++p) tma_load_3d(s + p * T8, &mq, 64 * p, h / a.hdiv, tok, b);
                bulk_load(s + NP * T8, fac + 2 * T8, T8, b);
            }
            // no copy outlives the CTA
            for (int c = max(chunks - 2, 0); c < chunks; ++c) {
                const int i = c & 1, ph = (c >> 1) & 1;
                wait(&bar.vt_full[i], ph, dead);
                wait(&bar.w_full[i], ph, dead);
                wait(&bar.k_full[i], ph, dead);
                wait(&bar.qp_full[i], ph, dead);
                wait(&bar.gates[c % kGateRing], (c / kGateRing) & 1, dead);
            }
        }
        __syncwarp();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
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

template <int DK>
rm_status launch(const Args& a, rm_dtype state_dt, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    if (!map_of(&mq, a.q, DK, a.H / a.hdiv, a.N, a.qs)) return fail("q", true);
    if (!map_of(&mk, a.k, DK, a.H / a.hdiv, a.N, a.ks)) return fail("k", true);
    if (!map_of(&mv, a.v, a.Dv, a.H, a.N, a.vs)) return fail("v", true);
    auto ff = gds_factor_kernel<DK>;
    if (!set_smem(ff, FactorSmem<DK>::bytes)) return fail("shared-memory attribute of the factors", false);
    ff<<<dim3(unsigned(chunk_slots(a)), unsigned(a.H)), 256, FactorSmem<DK>::bytes, s>>>(a, mq, mk);
    note_launch(1);
    if (!launch_ok()) return fail("launch of the factors", false);
    auto fw = state_dt == RM_F32 ? gds_walk_kernel<DK, float> : gds_walk_kernel<DK, __nv_bfloat16>;
    if (!set_smem(fw, WalkSmem<DK>::bytes)) return fail("shared-memory attribute of the walk", false);
    fw<<<dim3(unsigned((a.Dv + 127) / 128 * a.H), unsigned(a.S)), kWalkThreads, WalkSmem<DK>::bytes, s>>>(a, mq, mk, mv);
    note_launch(1);
    if (!launch_ok()) return fail("launch of the walk", false);
    return RM_OK;
}

}  // namespace

bool tc_supports(const Args& a, rm_dtype dt) {
    return dt == RM_BF16 && (a.Dk == 64 || a.Dk == 128) && a.max_len >= kChunkedLen && a.H <= 65535;
}

size_t tc_workspace_bytes(const Args& a) { return size_t(chunk_slots(a)) * a.H * factor_bytes(a.Dk); }

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
