// gds_kernels.cu -- the gated delta rule with a carried state as a token recurrence
// (rm_gdr_state_forward): decoding a few tokens for each of many sequences, and every shape
// that the chunked form on the tensor cores does not take.
//
// Per token, S in R^{Dk x Dv}:
//     d = beta (v - e^g S^T k),   o = scale (e^g S^T q + (q.k) d),   S <- e^g S + k d^T
// The columns of S are independent.  Bound by HBM when decoding: the state's read and write are
// nearly all of the traffic, and each is done once.
//
//   gds_token_kernel  in fp32.  A CTA owns 32 columns of one sequence's head and keeps them in
//                     registers over its tokens (Dk / 16 rows x 4 columns a thread, 128 threads); the
//                     state moves in 128-byte (fp32) pieces of a row.  One CTA per 32 columns keeps the
//                     loads in flight per thread to 32 registers and gives even one sequence of 16
//                     heads 32 or more CTAs.  Several tokens are taken four at a time, so that four share
//                     one pass over the state, one reduction across the threads and one update.
//                     256 sequences, one token, 16 heads of 128 x 128, fp32 state: 82 us, 6.6 TB/s.
//                     Ragged fp32 prompts of up to 301 tokens: 86 us, the latency of 75 tiles; one fp32
//                     prompt of 8192 tokens, 16 heads of 128 x 128: 4.4 ms.
//   gds_tile_kernel   bf16 inputs, four tokens as products of the warp's matrix instructions
#include <cstdio>
#include <type_traits>

#include "gds.cuh"

namespace rmcp {
namespace gds {

namespace {

constexpr int kCols = 32;      // columns of a CTA
constexpr int kTpb = 128;
constexpr unsigned kAllLanes = 0xffffffffu;

__device__ __forceinline__ void load4(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* x) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
    const float2 a = __bfloat1622float2(h[0]), b = __bfloat1622float2(h[1]);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
__device__ __forceinline__ void store4(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
    __nv_bfloat162 h[2] = {__floats2bfloat162_rn(x[0], x[1]), __floats2bfloat162_rn(x[2], x[3])};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
}

// The inputs of a tile of NT tokens, in fp32; keys and queries twice, as the factors of pairs.
template <int DK, int NT>
struct alignas(16) Tile {
    float2 q[NT][DK], k[NT][DK];
    float v[NT][kCols];
    float decay[NT], beta[NT];
    float kk[NT][NT], qk[NT][NT];  // k_t.k_r and q_t.k_r
};

// What a thread brings in of a tile: 16-byte units of q, k and v.  The loads of the next tile are
// issued before this one's tokens are taken and stored after them, so that a tile does not wait for
// memory.
template <typename T, int DK, int NT>
struct Fetch {
    static constexpr int E = 16 / sizeof(T);                // elements of a unit
    static constexpr int U = 2 * DK / E + kCols / E;        // units of a token
    static constexpr int N = (NT * U + kTpb - 1) / kTpb;    // units of a thread
    uint4 x[N];
    float gate;

    __device__ __forceinline__ void load(const Args& a, const T* q, const T* k, const T* v, const float* g, const float* beta, int t0,
                                         int n, int cols) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = threadIdx.x + i * kTpb, t = u / U, e = (u % U) * E;
            x[i] = make_uint4(0, 0, 0, 0);
            if (t >= n || t >= NT) continue;
            if (e < DK) x[i] = __ldg(reinterpret_cast<const uint4*>(q + (t0 + t) * a.qs[0] + e));
            else if (e < 2 * DK) x[i] = __ldg(reinterpret_cast<const uint4*>(k + (t0 + t) * a.ks[0] + e - DK));
            else if (e - 2 * DK < cols) x[i] = __ldg(reinterpret_cast<const uint4*>(v + (t0 + t) * a.vs[0] + e - 2 * DK));
        }
        const int t = threadIdx.x % NT;
        gate = 0.f;
        if (threadIdx.x < 2 * NT && t < n) gate = threadIdx.x < NT ? __ldg(g + (t0 + t) * a.gs) : __ldg(beta + (t0 + t) * a.bs);
    }

    __device__ __forceinline__ void store(Tile<DK, NT>& s) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = threadIdx.x + i * kTpb, t = u / U, e = (u % U) * E;
            if (t >= NT) continue;
            float y[E];
            if (sizeof(T) == 4) *reinterpret_cast<uint4*>(y) = x[i];
            else tc::unpack8(x[i], y);
            if (e < 2 * DK) {
                float2* to = e < DK ? s.q[t] + e : s.k[t] + e - DK;
#pragma unroll
                for (int j = 0; j < E; j += 2) *reinterpret_cast<float4*>(to + j) = make_float4(y[j], y[j], y[j + 1], y[j + 1]);
            } else {
#pragma unroll
                for (int j = 0; j < E; j += 4) *reinterpret_cast<float4*>(s.v[t] + e - 2 * DK + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
            }
        }
        if (threadIdx.x < NT) s.decay[threadIdx.x] = expf(gate);
        else if (threadIdx.x < 2 * NT) s.beta[threadIdx.x - NT] = gate;
    }
};

// N values of each lane, summed over the lanes that differ in bit `bit`, and shared between them: a
// lane keeps the first or the second half of them, by that bit.
template <int N>
__device__ __forceinline__ void halve(float* x, int bit) {
    const bool upper = threadIdx.x & bit;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float give = upper ? x[i] : x[N / 2 + i], keep = upper ? x[N / 2 + i] : x[i];
        x[i] = keep + __shfl_xor_sync(kAllLanes, give, bit);
    }
}

// A CTA: blockIdx.x = column block + blocks * head, blockIdx.y = sequence.  NT tokens at a time: their
// products with the state that the tile began with, one reduction, then the tile's own triangle
//     d_t = beta_t (v_t - G_t S^T k_t - sum_{r < t} G_t / G_r (k_t.k_r) d_r),   G_t = e^{g_0 + .. + g_t}
//     o_t = scale (G_t S^T q_t + sum_{r <= t} G_t / G_r (q_t.k_r) d_r)
// a column a lane, and one update of the state.
template <typename T, typename TS, int DK, int NT>
__global__ void __launch_bounds__(kTpb, NT == 1 ? 8 : 5) gds_token_kernel(const __grid_constant__ Args a) {
    constexpr int KR = DK / 16;  // rows of a thread: KR (tid / 8) ...
    constexpr int P = 8 * NT + 4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane & 7;
    const int blocks = (a.Dv + kCols - 1) / kCols;
    const int h = blockIdx.x / blocks, c0 = (blockIdx.x % blocks) * kCols;
    const int col = c0 + quad * 4, row = (tid >> 3) * KR;
    const bool live = col < a.Dv;  // Dv is a multiple of 8, a thread's columns of 4
    const Seq sq = sequence(a, blockIdx.y);
    const int cols = min(a.Dv - c0, kCols);
    zero_others(a, blockIdx.y, sq, static_cast<T*>(a.o) + int64_t(h) * a.Dv + c0, cols, tid, kTpb);
    if (sq.len <= 0 && !(sq.fresh && sq.slot >= 0)) return;  // a fresh empty sequence leaves a zero state
    T* o = static_cast<T*>(a.o) + (int64_t(sq.begin) * a.H + h) * a.Dv + c0;
    const int64_t os = int64_t(a.H) * a.Dv;
    if (sq.slot < 0) {  // padding
        zero_outputs(o, os, sq.len, cols, tid, kTpb);
        return;
    }
    TS* st = static_cast<TS*>(a.state) + ((int64_t(sq.slot) * a.H + h) * a.Dk + row) * a.Dv + col;
    uint64_t S[KR][2];  // pairs of columns
#pragma unroll
    for (int i = 0; i < KR; ++i) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (live && !sq.fresh) load4(st + i * a.Dv, x);
        S[i][0] = pair(x[0], x[1]), S[i][1] = pair(x[2], x[3]);
    }

    __shared__ Tile<DK, NT> tile;
    __shared__ __align__(16) float part[4][8][P];      // [warp][column quad][t][k | q][4]
    __shared__ __align__(16) float coef[4][NT][kCols]; // [warp][t][column]: d_t decayed to the tile's end
    const int hk = h / a.hdiv;
    const T* q = static_cast<const T*>(a.q) + sq.begin * a.qs[0] + hk * a.qs[1];
    const T* k = static_cast<const T*>(a.k) + sq.begin * a.ks[0] + hk * a.ks[1];
    const T* v = static_cast<const T*>(a.v) + sq.begin * a.vs[0] + h * a.vs[1] + c0;
    const float* g = a.g + sq.begin * a.gs + h;
    const float* beta = a.beta + sq.begin * a.bs + h;
    Fetch<T, DK, NT> next;
    if (sq.len > 0) next.load(a, q, k, v, g, beta, 0, sq.len, cols);
    for (int t0 = 0; t0 < sq.len; t0 += NT) {
        const int n = min(sq.len - t0, NT);
        next.store(tile);
        __syncthreads();
        if (t0 + NT < sq.len) next.load(a, q, k, v, g, beta, t0 + NT, sq.len - t0 - NT, cols);
        {  // the tile's products with the state
            uint64_t acc[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[t][c] = 0;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t < n) {
#pragma unroll
                    for (int i = 0; i < KR; ++i) {
                        const uint64_t kr = *reinterpret_cast<const uint64_t*>(&tile.k[t][row + i]), qr = *reinterpret_cast<const uint64_t*>(&tile.q[t][row + i]);
                        acc[t][0] = fma2(kr, S[i][0], acc[t][0]);
                        acc[t][1] = fma2(kr, S[i][1], acc[t][1]);
                        acc[t][2] = fma2(qr, S[i][0], acc[t][2]);
                        acc[t][3] = fma2(qr, S[i][1], acc[t][3]);
                    }
                }
            }
            float x[8 * NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t lo, hi;
                    unpair(acc[t][c], lo, hi);
                    x[8 * t + 2 * c] = __uint_as_float(lo), x[8 * t + 2 * c + 1] = __uint_as_float(hi);
                }
            halve<8 * NT>(x, 16);
            halve<4 * NT>(x, 8);
            float* to = part[warp][quad] + (lane >> 4) * 4 * NT + ((lane >> 3) & 1) * 2 * NT;
            if (NT == 1) {
                *reinterpret_cast<float2*>(to) = make_float2(x[0], x[1]);
            } else {
#pragma unroll
                for (int i = 0; i < 2 * NT; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            }
        }
        // k_t.k_r and q_t.k_r of one token a warp
        if (NT == 1) {
            if (warp == 0) {
                float x = 0.f;
#pragma unroll
                for (int e = 0; e < DK; e += 32)
                    if (DK >= 32 || lane < DK) x = fmaf(tile.q[0][e + lane].x, tile.k[0][e + lane].x, x);
                x = warp_sum(x);
                if (lane == 0) tile.qk[0][0] = x;
            }
        } else {
            float x[2 * NT];
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) x[i] = 0.f;
#pragma unroll
            for (int e = 0; e < DK; e += 32) {
                if (DK >= 32 || lane < DK) {
                    const float kt = tile.k[warp][e + lane].x, qt = tile.q[warp][e + lane].x;
#pragma unroll
                    for (int r = 0; r < NT; ++r) {
                        const float kr = tile.k[r][e + lane].x;
                        x[r] = fmaf(kt, kr, x[r]);
                        x[NT + r] = fmaf(qt, kr, x[NT + r]);
                    }
                }
            }
            halve<2 * NT>(x, 16);
            halve<NT>(x, 8);
            halve<NT / 2>(x, 4);
            x[0] += __shfl_xor_sync(kAllLanes, x[0], 2);
            x[0] += __shfl_xor_sync(kAllLanes, x[0], 1);
            if ((lane & 3) == 0) {
                const int at = lane >> 2;  // the three bits that chose the value
                (at < NT ? tile.kk : tile.qk)[warp][at % NT] = x[0];
            }
        }
        __syncthreads();
        float total = 1.f;  // G of the tile's last token
        {  // the tile's triangle: a column a lane, every warp the same; warp t stores token t
            float d[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                d[t] = 0.f;
                if (t < n) {
                    const float al = tile.decay[t];
                    total *= al;
                    float sk = 0.f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) sk += part[w][lane >> 2][8 * t + (lane & 3)];
                    float x = fmaf(-total, sk, tile.v[t][lane]);
#pragma unroll
                    for (int r = 0; r < t; ++r) {
                        d[r] *= al;
                        x = fmaf(-tile.kk[t][r], d[r], x);
                    }
                    d[t] = tile.beta[t] * x;
                    if (warp == t) {
                        float so = 0.f;
#pragma unroll
                        for (int w = 0; w < 4; ++w) so += part[w][lane >> 2][8 * t + 4 + (lane & 3)];
                        so *= total;
#pragma unroll
                        for (int r = 0; r <= t; ++r) so = fmaf(tile.qk[t][r], d[r], so);
                        if (lane < cols) o[(t0 + t) * os + lane] = from_f32<T>(a.scale * so);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) coef[warp][t][lane] = d[t];
            __syncwarp();
        }
        const uint64_t al = pair(total, total);
#pragma unroll
        for (int i = 0; i < KR; ++i) S[i][0] = mul2(al, S[i][0]), S[i][1] = mul2(al, S[i][1]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t < n) {
                const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(&coef[warp][t][4 * quad]);
#pragma unroll
                for (int i = 0; i < KR; ++i) {
                    const uint64_t kr = *reinterpret_cast<const uint64_t*>(&tile.k[t][row + i]);
                    S[i][0] = fma2(kr, d.x, S[i][0]);
                    S[i][1] = fma2(kr, d.y, S[i][1]);
                }
            }
        }
        if (t0 + NT < sq.len) __syncthreads();  // the tile has been read
    }
    if (live) {
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            uint32_t x[4];
            unpair(S[i][0], x[0], x[1]);
            unpair(S[i][1], x[2], x[3]);
            const float y[4] = {__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]), __uint_as_float(x[3])};
            store4(st + i * a.Dv, y);
        }
    }
}

// ---------------------------------------------------------------------------
// bf16 inputs, four tokens at a time as products of the warp's matrix instructions.  The four
// tokens' keys and queries are the eight columns of one m16n8k16 product with 16 value columns of
// the state as its rows, and the update of 16 values by 8 keys is one product over 16 = 4 tokens x 4
// parts.  (A product of the larger matrix unit has 64 rows or more and would leave through tensor
// memory; these tiles never leave the registers.)  A warp owns 16 or 32 value columns and all of
// Dk, so that no two warps meet; the lanes' rows and columns are permuted such that the state's
// elements are loaded and stored straight from the registers that enter the products.
//
// 61 sequences, four tokens, 32 heads of 128 x 256, bf16 state: 53.9 us, 4.9 TB/s, against 120 us of
// the fp32 recurrence, whose 1294 instructions for 4096 elements of state bound it.  What bounds it
// now is the latency of the state's reads at 12 warps an SM: 32 columns a warp (8 bytes a lane and
// row; 16 columns and 20 warps an SM: 78 us), everything else loaded before the state (after it:
// 64 us).  Longer calls keep the state in fp32 and 16 columns a warp, for twice the warps.  In a CUDA graph the
// same sequences take 50 us for four tokens, 102 for five to eight and 134 for twelve (32 columns a warp: 122 to 126,
// 158); with a fp32 state 79 for one token, 99 to 102 for two to four (152), 128 to 134 for five to eight (180).  One
// prompt of 32 tokens and 16 heads: 10 us (23).
//
// Keys and queries are bf16 and enter as they are.  A bf16 state enters its first tile as it is; a
// state in fp32, and d of a token, as the sum of three bf16, which hold its 24 bits.  Products
// accumulate in fp32.
// ---------------------------------------------------------------------------
// D += A B, bf16: A [16][16] by rows, B [16][8] by columns, D [16][8] fp32
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Row r of a lane's Dk / 4 rows of the state, less its first: runs of kRun rows go to the four lanes
// of a group in turn, so that they read a key side by side.
template <int DK>
struct Rows {
    static constexpr int kRun = DK < 32 ? DK / 4 : 8;
    static __device__ __forceinline__ constexpr int at(int r) { return r / kRun * 4 * kRun + r % kRun; }
};

// A lane's DK / 8 pairs of a key or query, or zeros
template <int DK>
__device__ __forceinline__ void load_pairs(const __nv_bfloat16* p, bool live, uint32_t* x) {
#pragma unroll
    for (int i = 0; i < DK / 8; ++i) x[i] = 0;
    if (!live) return;
    if (DK < 32) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        x[0] = u.x, x[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < DK / 8; i += 4) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p + Rows<DK>::at(2 * i)));
            x[i] = u.x, x[i + 1] = u.y, x[i + 2] = u.z, x[i + 3] = u.w;
        }
    }
}

// N adjacent words
template <int N>
__device__ __forceinline__ void load_words(const void* p, uint32_t* x) {
    if (N == 1) {
        x[0] = *static_cast<const uint32_t*>(p);
    } else if (N == 2) {
        const uint2 u = *static_cast<const uint2*>(p);
        x[0] = u.x, x[1] = u.y;
    } else {
        const uint4 u = *static_cast<const uint4*>(p);
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    }
}
template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t* x) {
    if (N == 1) *static_cast<uint32_t*>(p) = x[0];
    else if (N == 2) *static_cast<uint2*>(p) = make_uint2(x[0], x[1]);
    else *static_cast<uint4*>(p) = make_uint4(x[0], x[1], x[2], x[3]);
}

// The state of a warp, W times 16 columns: lane (g, t) = (lane / 4, lane % 4) holds columns 2W g ..
// 2W g + 2W - 1, two for each product, of its rows.  Element [w][b][c] is the pair of rows 2b, 2b + 1 of
// column 2w + c.  kPacked keeps the pairs of bf16 that were read: a state of one tile.
template <int DK, int W, bool kPacked>
struct TileState {
    using Pair = typename std::conditional<kPacked, uint32_t, uint64_t>::type;
    Pair x[W][DK / 8][2];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int b = 0; b < DK / 8; ++b) x[w][b][0] = x[w][b][1] = 0;
    }
    __device__ __forceinline__ void put(int w, int b, int c, uint32_t p) {
        if constexpr (kPacked) x[w][b][c] = p;
        else x[w][b][c] = widen2(p);
    }
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int Dv) {
#pragma unroll
        for (int b = 0; b < DK / 8; ++b) {
            uint32_t u[W], v[W];
            load_words<W>(p + Rows<DK>::at(2 * b) * Dv, u);
            load_words<W>(p + (Rows<DK>::at(2 * b) + 1) * Dv, v);
#pragma unroll
            for (int w = 0; w < W; ++w) put(w, b, 0, __byte_perm(u[w], v[w], 0x5410)), put(w, b, 1, __byte_perm(u[w], v[w], 0x7632));
        }
    }
    __device__ __forceinline__ void load(const float* p, int Dv) {
#pragma unroll
        for (int b = 0; b < DK / 8; ++b) {
            uint32_t u[2 * W], v[2 * W];
            load_words<2 * W>(p + Rows<DK>::at(2 * b) * Dv, u);
            load_words<2 * W>(p + (Rows<DK>::at(2 * b) + 1) * Dv, v);
#pragma unroll
            for (int w = 0; w < W; ++w) x[w][b][0] = pair(u[2 * w], v[2 * w]), x[w][b][1] = pair(u[2 * w + 1], v[2 * w + 1]);
        }
    }
    __device__ __forceinline__ uint64_t at(int w, int b, int c) const {
        if constexpr (kPacked) return widen2(x[w][b][c]);
        else return x[w][b][c];
    }
    // y += S^T [k; q], from the lane's pairs of the keys and queries
    __device__ __forceinline__ void product(const uint32_t* kq, float (*y)[4]) const {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            float z[2][4] = {};
#pragma unroll
            for (int s = 0; s < DK / 16; ++s) {
                if constexpr (kPacked) {
                    const uint32_t a[4] = {x[w][2 * s][0], x[w][2 * s][1], x[w][2 * s + 1][0], x[w][2 * s + 1][1]};
                    mma(s & 1 ? z[0] : y[w], a, kq[2 * s], kq[2 * s + 1]);
                } else {
                    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) split2(x[w][2 * s + i / 2][i % 2], hi[i], mid[i], lo[i]);
                    mma(z[1], lo, kq[2 * s], kq[2 * s + 1]);
                    mma(z[0], mid, kq[2 * s], kq[2 * s + 1]);
                    mma(y[w], hi, kq[2 * s], kq[2 * s + 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) y[w][i] += z[0][i] + z[1][i];
        }
    }
};

// Rows 2b and 2b + 1 of a lane's columns, each product's as it leaves: (column 0, rows), (column 1, rows)
template <int DK, int W>
__device__ __forceinline__ void store_rows(__nv_bfloat16* p, int b, int Dv, const float (*c)[4]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint32_t x[W];
#pragma unroll
        for (int w = 0; w < W; ++w) x[w] = pack2(c[w][e], c[w][2 + e]);
        store_words<W>(p + (Rows<DK>::at(2 * b) + e) * Dv, x);
    }
}
template <int DK, int W>
__device__ __forceinline__ void store_rows(float* p, int b, int Dv, const float (*c)[4]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint32_t x[2 * W];
#pragma unroll
        for (int w = 0; w < W; ++w) x[2 * w] = __float_as_uint(c[w][e]), x[2 * w + 1] = __float_as_uint(c[w][2 + e]);
        store_words<2 * W>(p + (Rows<DK>::at(2 * b) + e) * Dv, x);
    }
}

template <typename TS, int DK, int W, bool kPacked>
__global__ void __launch_bounds__(kTpb, 3) gds_tile_kernel(const __grid_constant__ Args a) {
    constexpr int NP = DK / 8, kRun = Rows<DK>::kRun;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int blocks = (a.Dv + 16 * W - 1) / (16 * W);
    const int unit = blockIdx.x * (kTpb / 32) + (threadIdx.x >> 5), h = unit / blocks;
    if (h >= a.H) return;
    const int col = unit % blocks * 16 * W + 2 * W * g;
    const bool live = col < a.Dv;  // Dv is a multiple of 8
    const Seq sq = sequence(a, blockIdx.y);
    const int64_t os = int64_t(a.H) * a.Dv;
    const int c0 = unit % blocks * 16 * W, cols = min(a.Dv - c0, 16 * W);
    zero_others(a, blockIdx.y, sq, static_cast<__nv_bfloat16*>(a.o) + int64_t(h) * a.Dv + c0, cols, lane, 32);
    if (sq.len <= 0 && !(sq.fresh && sq.slot >= 0)) return;  // a fresh empty sequence leaves a zero state
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + (int64_t(sq.begin) * a.H + h) * a.Dv + col;
    if (sq.slot < 0) {  // padding
        zero_outputs(o - 2 * W * g, os, sq.len, cols, lane, 32);
        return;
    }
    TS* st = static_cast<TS*>(a.state) + ((int64_t(sq.slot) * a.H + h) * a.Dk + kRun * t) * a.Dv + col;
    const int hk = h / a.hdiv;
    // this lane's key or query of a tile; the two keys of its terms of the update; its values
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + sq.begin * a.qs[0] + hk * a.qs[1];
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + sq.begin * a.ks[0] + hk * a.ks[1];
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + sq.begin * a.vs[0] + h * a.vs[1] + col;
    const int64_t kqs = g < 4 ? a.ks[0] : a.qs[0];
    const __nv_bfloat16* kq_row = (g < 4 ? k : q) + (g & 3) * kqs + kRun * t;
    const int i0 = 2 * (t & 1);  // the lane's tokens i0 and i0 + 1
    const __nv_bfloat16* up_row = k + i0 * a.ks[0] + kRun * (g >> 1);
    const uint32_t half = g & 1 ? 0x7632 : 0x5410;
    const float* gate = a.g + sq.begin * a.gs + h;
    const float* beta = a.beta + sq.begin * a.bs + h;

    uint32_t kq[NP], vx[4][W];
    float al1, be1;  // the gate and beta of token t
    auto fetch = [&](int t0) {
        const int n = sq.len - t0;
        load_pairs<DK>(kq_row + t0 * kqs, (g & 3) < n, kq);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int w = 0; w < W; ++w) vx[i][w] = 0;
            if (live && i < n) load_words<W>(v + (t0 + i) * a.vs[0], vx[i]);
        }
        al1 = t < n ? __ldg(gate + (t0 + t) * a.gs) : 0.f;
        be1 = t < n ? __ldg(beta + (t0 + t) * a.bs) : 0.f;
    };
    if (sq.len > 0) fetch(0);
    TileState<DK, W, kPacked> S;
    if (live && !sq.fresh) S.load(st, a.Dv);
    else S.zero();
    for (int t0 = 0; t0 < sq.len; t0 += 4) {
        const int n = min(sq.len - t0, 4);
        // y: columns 0 .. 3 of the product are S^T k, 4 .. 7 S^T q; kk: row i of them times column r
        float y[W][4] = {}, kk[4] = {};
        S.product(kq, y);
#pragma unroll
        for (int s = 0; s < DK / 16; ++s) {
            const uint32_t rows[4] = {kq[2 * s], 0u, kq[2 * s + 1], 0u};
            mma(kk, rows, kq[2 * s], kq[2 * s + 1]);
        }
        const float al_t = expf(al1), be_t = be1;
        uint64_t vf[4][W];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int w = 0; w < W; ++w) vf[i][w] = widen2(vx[i][w]);
        if (!kPacked && t0 + 4 < sq.len) fetch(t0 + 4);
        // the tile's triangle, every lane for its columns, two at a time
        uint64_t d[4][W], out[2][W];
        float total = 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float al = __shfl_sync(kAllLanes, al_t, i, 4), be = __shfl_sync(kAllLanes, be_t, i, 4);
            total *= al;
            const uint64_t al2 = pair(al, al), be2 = pair(be, be), to2 = pair(total, total), neg2 = pair(-total, -total);
            uint64_t x[W], z[W];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float s0 = __shfl_sync(kAllLanes, y[w][i & 1], i >> 1, 4), s1 = __shfl_sync(kAllLanes, y[w][2 + (i & 1)], i >> 1, 4);
                x[w] = fma2(neg2, pair(s0, s1), vf[i][w]);
                z[w] = mul2(to2, pair(y[w][i & 1], y[w][2 + (i & 1)]));  // lanes t >= 2: S^T q of i0 and i0 + 1
            }
#pragma unroll
            for (int r = 0; r < i; ++r) {
                const float kr = -__shfl_sync(kAllLanes, kk[r & 1], 4 * i + (r >> 1));
                const float qr = __shfl_sync(kAllLanes, kk[r & 1], 16 + 4 * i + (r >> 1));
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    d[r][w] = mul2(al2, d[r][w]);
                    x[w] = fma2(pair(kr, kr), d[r][w], x[w]);
                    z[w] = fma2(pair(qr, qr), d[r][w], z[w]);
                }
            }
            const float qi = __shfl_sync(kAllLanes, kk[i & 1], 16 + 4 * i + (i >> 1));
#pragma unroll
            for (int w = 0; w < W; ++w) {
                d[i][w] = mul2(be2, x[w]);
                z[w] = fma2(pair(qi, qi), d[i][w], z[w]);
                if (i < 2 || t & 1) out[i & 1][w] = z[w];
            }
        }
        if (t >= 2 && live) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t r[W];
#pragma unroll
                for (int w = 0; w < W; ++w) r[w] = pack2(mul2(pair(a.scale, a.scale), out[e][w]));
                if (i0 + e < n) store_words<W>(o + (t0 + i0 + e) * os, r);
            }
        }
        // the update, S <- G S + k d^T.  Terms 2t, 2t + 1 of a product are the first or second part of d of
        // the lane's tokens, terms 8 + 2t, 9 + 2t the third or nothing
        uint32_t da[W][4];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            uint32_t d0[2], d1[2], hi, mid, lo;
            unpair(t & 1 ? d[2][w] : d[0][w], d0[0], d0[1]);
            unpair(t & 1 ? d[3][w] : d[1][w], d1[0], d1[1]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                split2(pair(d0[c], d1[c]), hi, mid, lo);
                da[w][c] = t < 2 ? hi : mid;
                da[w][2 + c] = t < 2 ? lo : 0u;
            }
        }
        uint32_t ku[2][NP];
#pragma unroll
        for (int e = 0; e < 2; ++e) load_pairs<DK>(up_row + (t0 + e) * a.ks[0], i0 + e < n, ku[e]);
        const uint64_t al = pair(total, total);
#pragma unroll
        for (int b = 0; b < NP; ++b) {
            const uint32_t kb = __byte_perm(ku[0][b], ku[1][b], half);
            float c[W][4];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                uint32_t x[4];
                unpair(mul2(al, S.at(w, b, 0)), x[0], x[1]);
                unpair(mul2(al, S.at(w, b, 1)), x[2], x[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) c[w][i] = __uint_as_float(x[i]);
                mma(c[w], da[w], kb, kb);
                if constexpr (!kPacked) S.x[w][b][0] = pair(c[w][0], c[w][1]), S.x[w][b][1] = pair(c[w][2], c[w][3]);
            }
            if (kPacked && live) store_rows<DK, W>(st, b, a.Dv, c);
        }
        if (kPacked && t0 + 4 < sq.len) {  // a sequence longer than its bound: on from the state just stored
            fetch(t0 + 4);
            if (live) S.load(st, a.Dv);
        }
    }
    if (live && (!kPacked || sq.len <= 0)) {
#pragma unroll
        for (int b = 0; b < NP; ++b) {
            float c[W][4];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                uint32_t x[4];
                unpair(S.at(w, b, 0), x[0], x[1]);
                unpair(S.at(w, b, 1), x[2], x[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) c[w][i] = __uint_as_float(x[i]);
            }
            store_rows<DK, W>(st, b, a.Dv, c);
        }
    }
}

template <typename TS, int W, bool kPacked>
bool tile_launch(const Args& a, cudaStream_t s) {
    const int64_t units = int64_t((a.Dv + 16 * W - 1) / (16 * W)) * a.H;
    const dim3 grid(unsigned((units + kTpb / 32 - 1) / (kTpb / 32)), unsigned(a.S));
    auto f = a.Dk == 16   ? gds_tile_kernel<TS, 16, W, kPacked>
             : a.Dk == 32 ? gds_tile_kernel<TS, 32, W, kPacked>
             : a.Dk == 64 ? gds_tile_kernel<TS, 64, W, kPacked>
                          : gds_tile_kernel<TS, 128, W, kPacked>;
    f<<<grid, kTpb, 0, s>>>(a);
    note_launch(1);
    return launch_ok();
}

template <typename T, typename TS, int NT>
bool token_launch(const Args& a, cudaStream_t s) {
    const dim3 grid(unsigned((a.Dv + kCols - 1) / kCols * a.H), unsigned(a.S));
    auto f = a.Dk == 16   ? gds_token_kernel<T, TS, 16, NT>
             : a.Dk == 32 ? gds_token_kernel<T, TS, 32, NT>
             : a.Dk == 64 ? gds_token_kernel<T, TS, 64, NT>
                          : gds_token_kernel<T, TS, 128, NT>;
    f<<<grid, kTpb, 0, s>>>(a);
    note_launch(1);
    return launch_ok();
}

template <typename TS>
bool recurrence(const Args& a, bool f32, cudaStream_t s) {
    // Single tokens with a fp32 state: the token kernel, whose loads of 16 bytes a lane fill whole lines
    // (256 sequences, 16 heads of 128 x 128: 82 us; tiles: 98).  With a bf16 state: tiles (50 us; the
    // token kernel 64).
    const bool one = a.max_len <= 1;
    if (f32) return one ? token_launch<float, TS, 1>(a, s) : token_launch<float, TS, 4>(a, s);
    if constexpr (sizeof(TS) == 2) {
        if (a.max_len <= 4) return tile_launch<TS, 2, true>(a, s);
    } else {
        if (one) return token_launch<__nv_bfloat16, TS, 1>(a, s);
    }
    return tile_launch<TS, 1, false>(a, s);
}

rm_status check(const rm_gdr_state_problem* p, Args* a) {
    if (p == nullptr) return api_fail(RM_ERR_INVALID_ARG, "problem is null");
    if (p->num_seqs <= 0 || p->num_tokens < 0 || p->max_len < 0 || p->H <= 0 || p->qk_heads <= 0 || p->num_slots <= 0)
        return api_fail(RM_ERR_INVALID_ARG, "num_seqs, H, qk_heads and num_slots must be positive, num_tokens and max_len not negative");
    if (p->H % p->qk_heads) return api_fail(RM_ERR_INVALID_ARG, "qk_heads must divide H");
    if ((p->dtype != RM_F32 && p->dtype != RM_BF16) || (p->state_dtype != RM_F32 && p->state_dtype != RM_BF16))
        return api_fail(RM_ERR_INVALID_ARG, "dtype and state_dtype must be RM_F32 or RM_BF16");
    if (!(p->scale > -3.0e38f && p->scale < 3.0e38f)) return api_fail(RM_ERR_INVALID_ARG, "scale must be finite");
    if ((p->Dk != 16 && p->Dk != 32 && p->Dk != 64 && p->Dk != 128) || p->Dv <= 0 || p->Dv % 8 || p->Dv > 256)
        return api_fail(RM_ERR_UNSUPPORTED, "Dk must be in {16, 32, 64, 128}, Dv a multiple of 8 up to 256");
    if (p->num_seqs > 65535) return api_fail(RM_ERR_SHAPE, "num_seqs exceeds 65535");
    if (int64_t(p->H) * 8 > (int64_t(1) << 30)) return api_fail(RM_ERR_SHAPE, "H is too large");
    if (int64_t(p->num_tokens) > (int64_t(1) << 31) - 1 - 64 * 65536) return api_fail(RM_ERR_SHAPE, "num_tokens is too large");
    const int es = p->dtype == RM_F32 ? 4 : 2;
    for (int i = 0; i < 2; ++i) {
        // (a dimension of one element takes no step)
        const bool steps_qk = i ? p->qk_heads > 1 : p->num_tokens > 1, steps_v = i ? p->H > 1 : p->num_tokens > 1;
        if (p->q_stride[i] < int(steps_qk) || p->k_stride[i] < int(steps_qk) || p->v_stride[i] < int(steps_v))
            return api_fail(RM_ERR_INVALID_ARG, "the strides of q, k and v must be positive");
        if (p->q_stride[i] * es % 16 || p->k_stride[i] * es % 16 || p->v_stride[i] * es % 16)
            return api_fail(RM_ERR_ALIGNMENT, "the strides of q, k and v must be multiples of 16 bytes");
        a->qs[i] = p->q_stride[i], a->ks[i] = p->k_stride[i], a->vs[i] = p->v_stride[i];
    }
    if (p->g_stride < 0 || p->beta_stride < 0) return api_fail(RM_ERR_INVALID_ARG, "strides must not be negative");
    a->gs = p->g_stride, a->bs = p->beta_stride;
    // (no sequence is longer than all of them; no tokens at all: the recurrence, which needs none)
    a->max_len = p->max_len < p->num_tokens ? p->max_len : p->num_tokens;
    a->S = p->num_seqs, a->N = p->num_tokens, a->H = p->H, a->hdiv = p->H / p->qk_heads;
    a->Dk = p->Dk, a->Dv = p->Dv, a->slots_n = p->num_slots, a->scale = p->scale, a->each = 0;
    a->recurrent = p->recurrent != 0;
    return RM_OK;
}

rm_status element_aligned(const void* p, const char* name, int size) {
    char msg[96];
    if (p == nullptr || reinterpret_cast<uintptr_t>(p) % size) {
        std::snprintf(msg, sizeof(msg), "%s is %s", name, p ? "not aligned to its elements" : "NULL");
        return api_fail(p ? RM_ERR_ALIGNMENT : RM_ERR_INVALID_ARG, msg);
    }
    return RM_OK;
}

}  // namespace
}  // namespace gds
}  // namespace rmcp

#define RM_GDS_NEED(ptr)                            \
    do {                                            \
        rm_status s_ = rmcp::api_need((ptr), #ptr); \
        if (s_ != RM_OK) return s_;                 \
    } while (0)
#define RM_GDS_ELEM(ptr, size)                                           \
    do {                                                                 \
        rm_status s_ = rmcp::gds::element_aligned((ptr), #ptr, (size)); \
        if (s_ != RM_OK) return s_;                                      \
    } while (0)

extern "C" {

int32_t rm_gdr_state_path(const rm_gdr_state_problem* p) {
    rmcp::gds::Args a{};
    if (rmcp::gds::check(p, &a) != RM_OK) return -1;
    return rmcp::gds::tc_supports(a, p->dtype) ? 1 : 0;
}

size_t rm_gdr_state_workspace_size(const rm_gdr_state_problem* p) {
    rmcp::gds::Args a{};
    if (rmcp::gds::check(p, &a) != RM_OK) return 0;
    return rmcp::gds::tc_supports(a, p->dtype) ? rmcp::gds::tc_workspace_bytes(a) : 16;
}

rm_status rm_gdr_state_forward(const rm_gdr_state_problem* p, const void* q, const void* k, const void* v,
                               const float* g, const float* beta, const int32_t* cu_seqlens, const int32_t* slots,
                               const uint8_t* fresh, void* state, void* o, void* ws, rm_stream_t stream) {
    using namespace rmcp;
    gds::Args a{};
    rm_status st = gds::check(p, &a);
    if (st != RM_OK) return st;
    if (cu_seqlens == nullptr) {
        if (a.N % a.S) return api_fail(RM_ERR_SHAPE, "without cu_seqlens num_seqs must divide num_tokens");
        a.each = a.N / a.S;
        if (a.each > a.max_len) return api_fail(RM_ERR_SHAPE, "max_len is below the sequences' length");
    } else {
        RM_GDS_ELEM(cu_seqlens, 4);
    }
    if (slots == nullptr && a.S > a.slots_n) return api_fail(RM_ERR_SHAPE, "without slots num_seqs must not exceed num_slots");
    RM_GDS_NEED(state);
    if (a.N > 0) {
        RM_GDS_NEED(q);
        RM_GDS_NEED(k);
        RM_GDS_NEED(v);
        RM_GDS_ELEM(g, 4);
        RM_GDS_ELEM(beta, 4);
        RM_GDS_NEED(o);
    }
    if (slots != nullptr) RM_GDS_ELEM(slots, 4);
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.cu = cu_seqlens, a.slots = slots, a.fresh = fresh;
    a.state = state, a.o = o, a.ws = ws;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (gds::tc_supports(a, p->dtype)) {
        RM_GDS_NEED(ws);
        begin_launches();
        return gds::tc_launch(a, p->state_dtype, s);
    }
    begin_launches();
    const bool sf = p->state_dtype == RM_F32;
    const bool f32 = p->dtype == RM_F32;
    const bool ok = sf ? gds::recurrence<float>(a, f32, s) : gds::recurrence<__nv_bfloat16>(a, f32, s);
    if (ok) return RM_OK;
    char msg[256];
    std::snprintf(msg, sizeof(msg), "gated delta rule with a carried state: launch failed: %s", cuda_error_text());
    return api_fail(RM_ERR_CUDA, msg);
}

}  // extern "C"
