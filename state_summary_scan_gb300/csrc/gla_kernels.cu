// gla_kernels.cu -- linear attention with a decay for each head and a carried state as a token
// recurrence (rm_cp_gla_state_forward): decoding a few tokens for each of many sequences, and every
// shape that the chunked form on the tensor cores does not take.  (Several bf16 tokens go four at a
// time through the warp's matrix instructions: gds_kernels.cu.)
//
// Per token, S in R^{Dk x Dv}:
//     S <- e^g S + k v^T,   o = scale S^T q
// The columns of S are independent.  Bound by HBM when decoding: the state's read and write are
// nearly all of the traffic, and each is done once.
//
// A CTA owns 32 columns of one sequence's head and keeps them in registers over its tokens: a thread has
// 4 columns of Dk / 16 rows (two of 16), which it loads in pieces of 16 bytes (fp32).  It reads its own rows of q and k and its
// own columns of v straight from memory, the next tokens' before it takes these.  Arithmetic is fp32, on
// pairs of rows.  Tokens go NT at a time, whose outputs are summed across the threads at once.  256 sequences, one token, 16
// heads of 128 x 128, fp32 state: 82 us, 6.6 TB/s.
#include <cstdio>

#include "gla.cuh"

namespace rmcp {
namespace gla {

namespace {

constexpr int kCols = 32;  // columns of a CTA
constexpr unsigned kAllLanes = 0xffffffffu;

__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }

// N adjacent elements as they lie in memory; N * sizeof(T) is a multiple of 4.
template <typename T, int N>
struct Raw {
    static constexpr int W = N * int(sizeof(T)) / 4;
    uint32_t x[W];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (W == 1) {
            x[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
        } else if constexpr (W == 2) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
            x[0] = u.x, x[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
                x[i] = u.x, x[i + 1] = u.y, x[i + 2] = u.z, x[i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ uint64_t two(int i) const {  // elements 2i and 2i + 1
        if constexpr (sizeof(T) == 2) return widen2(x[i]);
        else return pair(x[2 * i], x[2 * i + 1]);
    }
};

__device__ __forceinline__ void load4(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* x) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float* x) { *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
}

// N values of each lane, summed over the lanes that differ in bit `bit`, and shared between them: a lane keeps
// the first or the second half of them, by that bit.
template <int N>
__device__ __forceinline__ void halve(float* x, int bit) {
    const bool upper = threadIdx.x & bit;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float give = upper ? x[i] : x[N / 2 + i], keep = upper ? x[N / 2 + i] : x[i];
        x[i] = keep + __shfl_xor_sync(kAllLanes, give, bit);
    }
}

constexpr int rows_of(int DK) { return DK >= 32 ? DK / 16 : 2; }
constexpr int threads_of(int DK) { return DK / rows_of(DK) * 8; }

// A thread's part of NT tokens
template <typename T, int KR, int NT>
struct Tokens {
    Raw<T, KR> q[NT], k[NT];
    Raw<T, 4> v[NT];
    float g[NT];
};

// A CTA: blockIdx.x = column block + blocks * head, blockIdx.y = sequence.
template <typename T, typename TS, int DK, int NT>
__global__ void __launch_bounds__(threads_of(DK), NT == 1 ? 8 : 4) gla_token_kernel(const __grid_constant__ Args a) {
    constexpr int KR = rows_of(DK), TPB = threads_of(DK), WARPS = TPB / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane & 7;
    const int blocks = (a.Dv + kCols - 1) / kCols;
    const int h = blockIdx.x / blocks, c0 = (blockIdx.x % blocks) * kCols;
    const int col = c0 + quad * 4, row = (tid >> 3) * KR;
    const bool live = col < a.Dv;  // Dv is a multiple of 8, a thread's columns of 4
    const int cols = min(a.Dv - c0, kCols);
    const Seq sq = sequence(a, blockIdx.y);
    zero_others(a, blockIdx.y, sq, static_cast<T*>(a.o) + int64_t(h) * a.Dv + c0, cols, tid, TPB);
    if (sq.len <= 0 && !(sq.fresh && sq.slot >= 0)) return;  // a fresh empty sequence leaves a zero state
    T* o = static_cast<T*>(a.o) + (int64_t(sq.begin) * a.H + h) * a.Dv + c0;
    const int64_t os = int64_t(a.H) * a.Dv;
    if (sq.slot < 0) {  // padding
        zero_outputs(o, os, sq.len, cols, tid, TPB);
        return;
    }
    const int hk = h / a.hdiv;
    const T* q = static_cast<const T*>(a.q) + sq.begin * a.qs[0] + hk * a.qs[1] + row;
    const T* k = static_cast<const T*>(a.k) + sq.begin * a.ks[0] + hk * a.ks[1] + row;
    const T* v = static_cast<const T*>(a.v) + sq.begin * a.vs[0] + h * a.vs[1] + (live ? col : 0);
    const float* g = a.g + sq.begin * a.gs + h;
    Tokens<T, KR, NT> next;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t0 + t < sq.len) {
                next.k[t].load(k + (t0 + t) * a.ks[0]);
                next.v[t].load(v + (t0 + t) * a.vs[0]);
                next.q[t].load(q + (t0 + t) * a.qs[0]);
                next.g[t] = __ldg(g + (t0 + t) * a.gs);
            }
        }
    };
    if (sq.len > 0) fetch(0);
    TS* st = static_cast<TS*>(a.state) + ((int64_t(sq.slot) * a.H + h) * DK + row) * a.Dv + col;
    uint64_t S[KR / 2][4];  // pairs of rows
#pragma unroll
    for (int i = 0; i < KR / 2; ++i) {
        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
        if (live && !sq.fresh) {
            load4(st + 2 * i * a.Dv, x);
            load4(st + (2 * i + 1) * a.Dv, y);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) S[i][c] = pair(x[c], y[c]);
    }

    // [warp][column quad][token of the quad's lanes][4]; two, so that a tile's sums are read while the next ones come
    __shared__ __align__(16) float part[2][WARPS][32][NT];
    for (int t0 = 0; t0 < sq.len; t0 += NT) {
        const int n = min(sq.len - t0, NT), b = (t0 / NT) & 1;
        const Tokens<T, KR, NT> now = next;
        if (t0 + NT < sq.len) fetch(t0 + NT);
        float x[4 * NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t < n) {
                // S + (e^g - 1) S near 1, where e^g itself has lost the bits that many tokens of a slow decay add up
                const bool near = now.g[t] > -0.7f && now.g[t] < 0.7f;
                const uint64_t al = both(near ? expm1f(now.g[t]) : expf(now.g[t]));
                uint64_t acc[4] = {0, 0, 0, 0}, vv[4];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t lo, hi;
                    unpair(now.v[t].two(c), lo, hi);
                    vv[2 * c] = pair(lo, lo), vv[2 * c + 1] = pair(hi, hi);
                }
#pragma unroll
                for (int i = 0; i < KR / 2; ++i) {
                    const uint64_t kk = now.k[t].two(i), qq = now.q[t].two(i);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        S[i][c] = fma2(kk, vv[c], near ? fma2(al, S[i][c], S[i][c]) : mul2(al, S[i][c]));
                        acc[c] = fma2(qq, S[i][c], acc[c]);
                    }
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t lo, hi;
                    unpair(acc[c], lo, hi);
                    x[4 * t + c] = __uint_as_float(lo) + __uint_as_float(hi);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) x[4 * t + c] = 0.f;
            }
        }
        // value i of a lane's 4 NT is that of token i / 4 and column i % 4; lane bits 4 and 3 choose a quarter
        halve<4 * NT>(x, 16);
        halve<2 * NT>(x, 8);
        float* to = part[b][warp][lane];
        if constexpr (NT % 4 == 0) {
#pragma unroll
            for (int i = 0; i < NT; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i) to[i] = x[i];
        }
        __syncthreads();
        for (int i = tid; i < n * kCols; i += TPB) {
            const int t = i / kCols, c = i % kCols, at = 4 * t + c % 4;  // value `at` of the quad c / 4
            const int from = at / NT * 8 + c / 4;                        // the lane that has it
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) y += part[b][w][from][at % NT];
            if (c < cols) o[(t0 + t) * os + c] = from_f32<T>(a.scale * y);
        }
    }
    if (live) {
#pragma unroll
        for (int i = 0; i < KR / 2; ++i) {
            float x[4], y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t lo, hi;
                unpair(S[i][c], lo, hi);
                x[c] = __uint_as_float(lo), y[c] = __uint_as_float(hi);
            }
            store4(st + 2 * i * a.Dv, x);
            store4(st + (2 * i + 1) * a.Dv, y);
        }
    }
}

// ---------------------------------------------------------------------------
// Prompts in chunks of 32 tokens in fp32 arithmetic: fp32 tokens, and bf16 ones of shapes that the tensor cores do not take.  With b_t the running sum of a chunk's gates and S the state before it:
//     o_t = scale (e^{b_t} S^T q_t + sum_{s <= t} e^{b_t - b_s} (q_t.k_s) v_s),   S <- e^{b_31} S + sum_s e^{b_31 - b_s} k_s v_s^T
// A CTA has 32 columns of a sequence's head.  The products are plain fp32 multiply-adds on tiles in shared memory, two tokens x
// four columns (of scores, of outputs) or Dk / 16 rows x four columns (of the state) a thread, the next chunk's tokens on
// their way meanwhile.  What bounds it is the multiply-adds and, in short sequences, the three barriers of a chunk; the
// recurrence, which it replaces, pays the latency of a barrier every four tokens (7 prompts of up to 301 tokens, 6 heads of 32 x
// 40: 35 us, the recurrence 53; one of 2048, 16 heads of 128 x 128: 371 and 610).
// ---------------------------------------------------------------------------
constexpr int kTokens = 32;
// Tokens of the longest sequence from which it is taken.  us in a CUDA graph, recurrence / chunks:
//     tokens                               12           16           24           64
//     one sequence, 16 heads of 128 x 128  11.0 / 7.8   14.3 / 7.8   20.8 / 7.8   53 / 13
//     64 sequences, 16 heads of 64 x 64    31 / 46      39 / 47      55 / 48      138 / 86
//     7 sequences, 6 heads of 32 x 40      3.8 / 4.9    4.5 / 5.0    5.9 / 4.9    12.3 / 8.1
//     61 sequences, 16 heads of 128 x 128  147 / 149    191 / 149    280 / 151    723 / 272
constexpr int kTokenLen = 20;
template <int DK>
struct ChunkSmem {
    static constexpr int row = DK + 4;  // (rows of 16 keys side by side lie in different banks)
    struct In {
        float q[kTokens][row], k[kTokens][row], v[kTokens][kCols];
    } in[2];
    float S[DK][kCols];
    float P[kTokens][kTokens + 4];
    float out[kTokens], dec[kTokens], hi[kTokens], lo[kTokens];  // scale e^{b_t}, e^{b_31 - b_t}, b_t in two parts
    float end;
    int near;
};
__device__ __forceinline__ void copy16(float* to, const float* from, bool live) {  // zeros where it is not live
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(to)), "l"(from), "r"(live ? 16 : 0) : "memory");
}

template <typename T, typename TS, int DK>
__global__ void __launch_bounds__(128) gla_chunk_kernel(const __grid_constant__ Args a) {
    // tokens of a thread (one, and 256 threads: 2048 tokens of 16 heads of 128 x 128 456 us for 382, 8 prompts of 300 of 64 x
    // 64 82 for 60), and rows
    constexpr int TOK = 2, TPB = 256 / TOK, KR = DK / 16;
    using L = ChunkSmem<DK>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    L& sm = *reinterpret_cast<L*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = tid & 7, t0 = TOK * (tid >> 3), row = (tid >> 3) * KR;
    const int blocks = (a.Dv + kCols - 1) / kCols;
    const int h = blockIdx.x / blocks, c0 = (blockIdx.x % blocks) * kCols, col = c0 + quad * 4;
    const bool live = col < a.Dv;  // Dv is a multiple of 8, a thread's columns of 4
    const int cols = min(a.Dv - c0, kCols);
    const Seq sq = sequence(a, blockIdx.y);
    zero_others(a, blockIdx.y, sq, static_cast<T*>(a.o) + int64_t(h) * a.Dv + c0, cols, tid, TPB);
    if (sq.len <= 0 && !(sq.fresh && sq.slot >= 0)) return;  // a fresh empty sequence leaves a zero state
    T* o = static_cast<T*>(a.o) + (int64_t(sq.begin) * a.H + h) * a.Dv + c0;
    const int64_t os = int64_t(a.H) * a.Dv;
    if (sq.slot < 0) {  // padding
        zero_outputs(o, os, sq.len, cols, tid, TPB);
        return;
    }
    const int hk = h / a.hdiv;
    const T* q = static_cast<const T*>(a.q) + sq.begin * a.qs[0] + hk * a.qs[1];
    const T* k = static_cast<const T*>(a.k) + sq.begin * a.ks[0] + hk * a.ks[1];
    const T* v = static_cast<const T*>(a.v) + sq.begin * a.vs[0] + h * a.vs[1] + c0;
    const float* g = a.g + sq.begin * a.gs + h;
    // A chunk's tokens; those past the end are zeros.  fp32 is copied into shared memory as it is; bf16 is read into
    // registers, and put there as fp32 when the chunk before has been taken.
    constexpr bool kCopy = sizeof(T) == 4;
    constexpr int NQ = kTokens * DK / 8 / TPB > 0 ? kTokens * DK / 8 / TPB : 1;  // units of eight of q, and of k, a thread
    Raw<T, 8> raw[kCopy ? 1 : 2 * NQ + 1];
    auto fetch = [&](int from) {
        if constexpr (kCopy) {
            typename L::In& to = sm.in[(from / kTokens) & 1];
            for (int u = tid; u < kTokens * (DK / 4); u += TPB) {
                const int t = u / (DK / 4), e = u % (DK / 4) * 4;
                const bool there = from + t < sq.len;
                copy16(&to.q[t][e], q + (there ? from + t : 0) * a.qs[0] + e, there);
                copy16(&to.k[t][e], k + (there ? from + t : 0) * a.ks[0] + e, there);
            }
            for (int u = tid; u < kTokens * (kCols / 4); u += TPB) {
                const int t = u / (kCols / 4), e = u % (kCols / 4) * 4;
                const bool there = from + t < sq.len && e < cols;
                copy16(&to.v[t][e], v + (there ? (from + t) * a.vs[0] + e : 0), there);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else {
#pragma unroll
            for (int i = 0; i <= 2 * NQ; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w) raw[i].x[w] = 0;
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const int u = tid + i * TPB, t = u / (DK / 8), e = u % (DK / 8) * 8;
                if (t < kTokens && from + t < sq.len) {
                    raw[i].load(q + (from + t) * a.qs[0] + e);
                    raw[NQ + i].load(k + (from + t) * a.ks[0] + e);
                }
            }
            const int t = tid / (kCols / 8), e = tid % (kCols / 8) * 8;  // (32 x 32 values: one unit a thread)
            if (from + t < sq.len && e < cols) raw[2 * NQ].load(v + (from + t) * a.vs[0] + e);
        }
    };
    auto place = [&](int from) {  // what fetch() read
        if constexpr (!kCopy) {
            typename L::In& to = sm.in[(from / kTokens) & 1];
            auto put = [](float* p, const Raw<T, 8>& r) {
#pragma unroll
                for (int w = 0; w < 4; w += 2)
                    *reinterpret_cast<ulonglong2*>(p + 2 * w) = make_ulonglong2(r.two(w), r.two(w + 1));
            };
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const int u = tid + i * TPB, t = u / (DK / 8), e = u % (DK / 8) * 8;
                if (t < kTokens) {
                    put(&to.q[t][e], raw[i]);
                    put(&to.k[t][e], raw[NQ + i]);
                }
            }
            put(&to.v[tid / (kCols / 8)][tid % (kCols / 8) * 8], raw[2 * NQ]);
        }
    };
    auto gate = [&](int from) { return warp == 0 && from + lane < sq.len ? __ldg(g + (from + lane) * a.gs) : 0.f; };
    if (sq.len > 0) {
        fetch(0);
        place(0);
    }
    float next = gate(0);
    TS* st = static_cast<TS*>(a.state) + ((int64_t(sq.slot) * a.H + h) * DK + row) * a.Dv + col;
    float S[KR][4];
#pragma unroll
    for (int i = 0; i < KR; ++i) {
#pragma unroll
        for (int c = 0; c < 4; ++c) S[i][c] = 0.f;
        if (live && !sq.fresh) load4(st + i * a.Dv, S[i]);
        store4(&sm.S[row + i][4 * quad], S[i]);
    }
    for (int from = 0; from < sq.len; from += kTokens) {
        const typename L::In& in = sm.in[(from / kTokens) & 1];
        const int n = min(sq.len - from, kTokens);
        if (kCopy) asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the tokens and the state are there, the other tokens and P have been used
        if (from + kTokens < sq.len) fetch(from + kTokens);
        if (warp == 0) {  // the gates: a token a lane, sums held as two floats
            float x = next, y = 0.f;
            next = gate(from + kTokens);
            x = x < -110.f ? -110.f : x;  // (e^-110 is 0)
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const float u = __shfl_up_sync(kAllLanes, x, s), w = __shfl_up_sync(kAllLanes, y, s);
                if (lane >= s) {
                    const float sum = x + u, z = sum - x;
                    y += w + ((x - (sum - z)) + (u - z));
                    x = sum;
                }
            }
            const float ex = __shfl_sync(kAllLanes, x, 31), ey = __shfl_sync(kAllLanes, y, 31), e = ex + ey;
            sm.out[lane] = a.scale * expf(x + y);
            sm.dec[lane] = expf((ex - x) + (ey - y));
            sm.hi[lane] = x, sm.lo[lane] = y;
            if (lane == 0) {
                sm.near = e > -0.7f && e < 0.7f;  // near 1 the decay as its distance from 1 (see gla_token_kernel)
                sm.end = sm.near ? expm1f(e) : expf(e);
            }
        }
        float x[TOK][4];  // scores of the thread's tokens with quad + 8 j
#pragma unroll
        for (int i = 0; i < TOK; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll 4
        for (int e = 0; e < DK; e += 4) {
            float4 u[TOK];
#pragma unroll
            for (int i = 0; i < TOK; ++i) u[i] = *reinterpret_cast<const float4*>(&in.q[t0 + i][e]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 y = *reinterpret_cast<const float4*>(&in.k[quad + 8 * j][e]);
#pragma unroll
                for (int i = 0; i < TOK; ++i) x[i][j] = fmaf(u[i].w, y.w, fmaf(u[i].z, y.z, fmaf(u[i].y, y.y, fmaf(u[i].x, y.x, x[i][j]))));
            }
        }
        __syncthreads();  // the gates are there
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
            const float bh = sm.hi[t0 + i], bl = sm.lo[t0 + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int s = quad + 8 * j;
                sm.P[t0 + i][s] = s <= t0 + i ? a.scale * x[i][j] * expf((bh - sm.hi[s]) + (bl - sm.lo[s])) : 0.f;
            }
        }
        float y[TOK][4];
#pragma unroll
        for (int i = 0; i < TOK; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) y[i][c] = 0.f;
        auto product = [&](const float* l, int stride, const float* m, int count) {  // y += l m, four terms at a time
#pragma unroll 4
            for (int e = 0; e < count; e += 4) {
                float u[TOK][4];
#pragma unroll
                for (int i = 0; i < TOK; ++i) load4(l + i * stride + e, u[i]);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float r[4];
                    load4(m + (e + b) * kCols + 4 * quad, r);
#pragma unroll
                    for (int i = 0; i < TOK; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) y[i][c] = fmaf(u[i][b], r[c], y[i][c]);
                }
            }
        };
        product(in.q[t0], L::row, sm.S[0], DK);
#pragma unroll
        for (int i = 0; i < TOK; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) y[i][c] *= sm.out[t0 + i];
        __syncthreads();  // P is there, and the state has been read
        product(sm.P[t0], kTokens + 4, in.v[0], (t0 + TOK + 3) / 4 * 4);
#pragma unroll
        for (int i = 0; i < TOK; ++i)
            if (live && t0 + i < n) store4(o + (from + t0 + i) * os + 4 * quad, y[i]);
        if (from + kTokens < sq.len) place(from + kTokens);
        const float end = sm.end;
        if (sm.near) {
#pragma unroll
            for (int i = 0; i < KR; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) S[i][c] = fmaf(end, S[i][c], S[i][c]);
        } else {
#pragma unroll
            for (int i = 0; i < KR; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) S[i][c] *= end;
        }
        float w[KR][4];  // summed by itself: the state's bits are rounded once a chunk
#pragma unroll
        for (int i = 0; i < KR; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) w[i][c] = 0.f;
#pragma unroll 4
        for (int s = 0; s < kTokens; ++s) {  // (past the end keys and values are zeros)
            float r[4], ks[KR];
            load4(&in.v[s][4 * quad], r);
            const float d = sm.dec[s];
            if constexpr (KR >= 4) {
#pragma unroll
                for (int i = 0; i < KR; i += 4) load4(&in.k[s][row + i], ks + i);
            } else {
#pragma unroll
                for (int i = 0; i < KR; ++i) ks[i] = in.k[s][row + i];
            }
#pragma unroll
            for (int i = 0; i < KR; ++i) {
                const float x = ks[i] * d;
#pragma unroll
                for (int c = 0; c < 4; ++c) w[i][c] = fmaf(x, r[c], w[i][c]);
            }
        }
#pragma unroll
        for (int i = 0; i < KR; ++i) {
#pragma unroll
            for (int c = 0; c < 4; ++c) S[i][c] += w[i][c];
            store4(&sm.S[row + i][4 * quad], S[i]);
        }
    }
    if (live) {
#pragma unroll
        for (int i = 0; i < KR; ++i) store4(st + i * a.Dv, S[i]);
    }
}

template <typename T, typename TS>
bool chunk_launch(const Args& a, cudaStream_t s) {
    const dim3 grid(unsigned((a.Dv + kCols - 1) / kCols * a.H), unsigned(a.S));
    auto run = [&](auto f, size_t bytes) {
        if (!tc::set_smem(f, bytes)) return false;
        f<<<grid, 128, bytes, s>>>(a);
        note_launch(1);
        return launch_ok();
    };
    return a.Dk == 16   ? run(gla_chunk_kernel<T, TS, 16>, sizeof(ChunkSmem<16>))
           : a.Dk == 32 ? run(gla_chunk_kernel<T, TS, 32>, sizeof(ChunkSmem<32>))
           : a.Dk == 64 ? run(gla_chunk_kernel<T, TS, 64>, sizeof(ChunkSmem<64>))
                        : run(gla_chunk_kernel<T, TS, 128>, sizeof(ChunkSmem<128>));
}

template <typename T, typename TS, int NT>
bool token_launch(const Args& a, cudaStream_t s) {
    const dim3 grid(unsigned((a.Dv + kCols - 1) / kCols * a.H), unsigned(a.S));
    auto run = [&](auto f, int DK) { f<<<grid, threads_of(DK), 0, s>>>(a); };
    if (a.Dk == 16) run(gla_token_kernel<T, TS, 16, NT>, 16);
    else if (a.Dk == 32) run(gla_token_kernel<T, TS, 32, NT>, 32);
    else if (a.Dk == 64) run(gla_token_kernel<T, TS, 64, NT>, 64);
    else run(gla_token_kernel<T, TS, 128, NT>, 128);
    note_launch(1);
    return launch_ok();
}

template <typename T, typename TS>
bool recurrence(const Args& a, cudaStream_t s) {
    // (bf16 with 64 rows and more is in chunks on the tensor cores from 32 or 64 tokens)
    if (!a.recurrent && a.max_len >= kTokenLen && (sizeof(T) == 4 || a.Dk < 64)) return chunk_launch<T, TS>(a, s);
    if constexpr (sizeof(T) == 4) {
        return a.max_len <= 1 ? token_launch<T, TS, 1>(a, s) : token_launch<T, TS, 4>(a, s);
    } else {
        // Single tokens: the token kernel, but tiles for a bf16 state of 128 rows (256 sequences of 16 heads of 128 x 128: fp32
        // 81 us and tiles 93, bf16 53 and tiles 48; 64 of 64 x 64, bf16: 6.5 and tiles 7.1).  Several: tiles (61 sequences,
        // four tokens, 32 heads of 128 x 256, bf16 state: 48 us, the token kernel 96; fp32 state: 108 us).
        const bool tiles = a.max_len > 1 || (sizeof(TS) == 2 && a.Dk == 128);
        return tiles ? gds::plain_tiles(a, sizeof(TS) == 4 ? RM_F32 : RM_BF16, s) : token_launch<T, TS, 1>(a, s);
    }
}

}  // namespace
}  // namespace gla
}  // namespace rmcp

#define RM_GLA_NEED(ptr)                            \
    do {                                            \
        rm_status s_ = rmcp::api_need((ptr), #ptr); \
        if (s_ != RM_OK) return s_;                 \
    } while (0)
#define RM_GLA_ELEM(ptr, size)                                           \
    do {                                                                 \
        rm_status s_ = rmcp::gds::element_aligned((ptr), #ptr, (size)); \
        if (s_ != RM_OK) return s_;                                      \
    } while (0)

extern "C" {

int32_t rm_cp_gla_state_path(const rm_gdr_state_problem* p) {
    rmcp::gla::Args a{};
    if (rmcp::gds::check(p, &a) != RM_OK) return -1;
    return rmcp::gla::tc_supports(a, p->dtype) ? 1 : 0;
}

size_t rm_cp_gla_state_workspace_size(const rm_gdr_state_problem* p) {
    rmcp::gla::Args a{};
    if (rmcp::gds::check(p, &a) != RM_OK) return 0;
    return rmcp::gla::tc_supports(a, p->dtype) ? rmcp::gla::tc_workspace_bytes(a) : 16;
}

rm_status rm_cp_gla_state_forward(const rm_gdr_state_problem* p, const void* q, const void* k, const void* v, const float* g,
                               const int32_t* cu_seqlens, const int32_t* slots, const uint8_t* fresh, void* state, void* o,
                               void* ws, rm_stream_t stream) {
    using namespace rmcp;
    gla::Args a{};
    rm_status st = gds::check(p, &a);
    if (st != RM_OK) return st;
    if (cu_seqlens == nullptr) {
        if (a.N % a.S) return api_fail(RM_ERR_SHAPE, "without cu_seqlens num_seqs must divide num_tokens");
        a.each = a.N / a.S;
        if (a.each > a.max_len) return api_fail(RM_ERR_SHAPE, "max_len is below the sequences' length");
    } else {
        RM_GLA_ELEM(cu_seqlens, 4);
    }
    if (slots == nullptr && a.S > a.slots_n) return api_fail(RM_ERR_SHAPE, "without slots num_seqs must not exceed num_slots");
    RM_GLA_NEED(state);
    if (a.N > 0) {
        RM_GLA_NEED(q);
        RM_GLA_NEED(k);
        RM_GLA_NEED(v);
        RM_GLA_ELEM(g, 4);
        RM_GLA_NEED(o);
    }
    if (slots != nullptr) RM_GLA_ELEM(slots, 4);
    // Heads and sequences are taken in no order: what one writes, another must not read
    const int64_t es = p->dtype == RM_F32 ? 4 : 2, tokens = a.N;
    const int64_t o_bytes = tokens * a.H * a.Dv * es, st_bytes = int64_t(a.slots_n) * a.H * a.Dk * a.Dv * (p->state_dtype == RM_F32 ? 4 : 2);
    auto apart = [](const void* x, int64_t xb, const void* y, int64_t yb) {
        const uintptr_t i = reinterpret_cast<uintptr_t>(x), j = reinterpret_cast<uintptr_t>(y);
        return x == nullptr || y == nullptr || i + uint64_t(xb) <= j || j + uint64_t(yb) <= i;
    };
    auto reach = [&](const int64_t* steps, int heads, int n) { return ((tokens - 1) * steps[0] + (heads - 1) * steps[1] + n) * es; };
    if (tokens > 0) {
        const int qk = a.H / a.hdiv;
        const struct { const void* at; int64_t bytes; } in[] = {{q, reach(a.qs, qk, a.Dk)}, {k, reach(a.ks, qk, a.Dk)}, {v, reach(a.vs, a.H, a.Dv)},
                                                                {g, ((tokens - 1) * a.gs + a.H) * 4}};
        bool ok = apart(o, o_bytes, state, st_bytes);
        for (const auto& x : in) ok = ok && apart(o, o_bytes, x.at, x.bytes) && apart(state, st_bytes, x.at, x.bytes);
        if (!ok) return api_fail(RM_ERR_INVALID_ARG, "o or the state overlaps another tensor");
    }
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = nullptr, a.cu = cu_seqlens, a.slots = slots, a.fresh = fresh;
    a.state = state, a.o = o, a.ws = ws;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool sf = p->state_dtype == RM_F32;
    if (gla::tc_supports(a, p->dtype)) {
        RM_GLA_NEED(ws);
        begin_launches();
        return gla::tc_launch(a, p->state_dtype, s);
    }
    begin_launches();
    bool ok;
    if (p->dtype == RM_F32) ok = sf ? gla::recurrence<float, float>(a, s) : gla::recurrence<float, __nv_bfloat16>(a, s);
    else ok = sf ? gla::recurrence<__nv_bfloat16, float>(a, s) : gla::recurrence<__nv_bfloat16, __nv_bfloat16>(a, s);
    if (ok) return RM_OK;
    char msg[256];
    std::snprintf(msg, sizeof(msg), "linear attention with a carried state: launch failed: %s", cuda_error_text());
    return api_fail(RM_ERR_CUDA, msg);
}

}  // extern "C"
