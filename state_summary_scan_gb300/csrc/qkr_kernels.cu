// qkr_kernels.cu -- the norm of each head of queries and keys and the position
// rotation in one pass, forward and backward (rm_cp_qkr_*).
//
// Per head row x in R^D with weight w (optional), table row (c, s) of the token's position:
//     r = (sum x^2 / D + eps)^(-1/2)  (rms)  |  (sum x^2 + eps)^(-1/2)  (l2)  |  1  (none)
//     y = x r w;   for each pair (a, b) of the first R elements: a' = y_a c - y_b s, b' = y_b c + y_a s
// Backward, with d the incoming gradient turned back by the transposed rotation:
//     dw = sum over rows of d x r,   u = d w,   dx = r u - r^3 x (sum u x) / D   (l2: no / D)
//
// Bound by HBM: the forward reads and writes every row once; the backward reads the gradient
// and the row and writes one.  A row is spread over D/8 lanes (16 bytes of bf16 a lane), so the
// sums of a row are a few shuffles and nothing is staged in shared memory; in the half layout
// the partner of a lane's eight elements is the eight elements of the lane R/16 away.  A warp
// keeps one token's cos and sin in registers over that token's heads.
#include <cstdio>

#include "tc_tiles.cuh"

namespace rmcp {
namespace qkr {

using tc::pack8;
using tc::unpack8;

namespace {

constexpr int kWarps = 8;
constexpr unsigned kAll = 0xffffffffu;

struct Args {
    int B, T, Hq, Hk, D, R, norm, inter;
    float eps;
    int max_pos, pos_rows, pos64;
    int64_t qs[3], ks[3];   // row, token, head strides of q and k (elements)
    int split;              // warps of a token: each takes every split-th group of heads
    const void* q;
    const void* k;
    const float* wq;
    const float* wk;
    const float* table;
    const void* pos;
    void* qo;               // forward: q', k'; backward: dq, dk
    void* ko;
    const void* gq;         // backward: gradients of q', k'
    const void* gk;
    float* part;            // backward: [blocks][2][D] partial weight gradients
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(p)), x);
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* x) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint4*>(p) = pack8(x);
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Sum over the LANES lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}

// Position of token t of row b; -1 where it lies outside the table.
__device__ __forceinline__ int position(const Args& a, int b, int t) {
    if (a.pos == nullptr) return t < a.max_pos ? t : -1;
    const int64_t i = (a.pos_rows > 1 ? int64_t(b) * a.T : 0) + t;
    const int64_t p = a.pos64 ? __ldg(static_cast<const long long*>(a.pos) + i)
                              : int64_t(__ldg(static_cast<const int*>(a.pos) + i));
    return p >= 0 && p < a.max_pos ? int(p) : -1;
}

// The rotation of a lane's eight elements e0 .. e0 + 7, of which those below R turn.
// kFast: R is a multiple of 16 (half layout) or 8 (interleaved), so a lane's elements turn
// together and their partners sit in one lane; otherwise each element finds its own partner
// through the warp's row buffer.
template <int LANES, bool kInter, bool kFast>
struct Turn {
    float c[kInter && kFast ? 4 : 8], s[kInter && kFast ? 4 : 8];
    bool on;       // kFast: the lane's elements turn
    int from;      // kFast, half: the partner's lane

    __device__ __forceinline__ void load(const Args& a, int b, int t, int e0, int lane) {
        on = false;
        from = lane;
#pragma unroll
        for (int i = 0; i < int(sizeof(c) / 4); ++i) c[i] = 1.f, s[i] = 0.f;
        if (a.R == 0) return;
        const int p = position(a, b, t), h = a.R / 2;
        const float* row = a.table + int64_t(p < 0 ? 0 : p) * a.R;
        if (kFast) {
            if (e0 >= a.R) return;
            on = true;
            const int n = kInter ? 4 : 8, at = kInter ? e0 / 2 : (e0 < h ? e0 : e0 - h);
#pragma unroll
            for (int i = 0; i < n; i += 4) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(row + at + i));
                const float4 y = __ldg(reinterpret_cast<const float4*>(row + h + at + i));
                c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
                s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
            }
            if (!kInter) {
                from = e0 < h ? lane + h / 8 : lane - h / 8;
                if (e0 < h) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[i] = -s[i];
                }
            }
        } else {
            // the second member of a pair adds s times the first, the first subtracts
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i;
                if (e >= a.R) continue;
                const int at = kInter ? e / 2 : (e < h ? e : e - h);
                const bool first = kInter ? !(e & 1) : e < h;
                c[i] = __ldg(row + at);
                s[i] = first ? -__ldg(row + h + at) : __ldg(row + h + at);
            }
        }
        if (p < 0) {  // a position outside the table: its rotated elements are NaN
#pragma unroll
            for (int i = 0; i < int(sizeof(c) / 4); ++i)
                if (kFast || e0 + i < a.R) c[i] = __int_as_float(0x7fffffff);
        }
    }

    // y <- rotation of y (kBack: of the transposed rotation).  Whole-warp call.
    template <bool kBack>
    __device__ __forceinline__ void apply(const Args& a, int e0, float* y, float* buf) const {
        if (kFast && kInter) {
            if (!on) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = y[2 * i], v = y[2 * i + 1], t = kBack ? -s[i] : s[i];
                y[2 * i] = u * c[i] - v * t;
                y[2 * i + 1] = v * c[i] + u * t;
            }
        } else if (kFast) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float o = __shfl_sync(kAll, y[i], from);
                const float z = kBack ? y[i] * c[i] - o * s[i] : y[i] * c[i] + o * s[i];
                y[i] = on ? z : y[i];
            }
        } else {
            const int h = a.R / 2;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) buf[i] = y[i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i;
                if (e >= a.R) continue;
                const int o = kInter ? (e ^ 1) : (e < h ? e + h : e - h);
                const float p = buf[o - e0];
                y[i] = kBack ? y[i] * c[i] - p * s[i] : y[i] * c[i] + p * s[i];
            }
        }
    }
};

__device__ __forceinline__ float norm_scale(const Args& a, float sq) {
    return a.norm == 0 ? 1.f : rsqrtf((a.norm == 1 ? sq / float(a.D) : sq) + a.eps);
}

template <int LANES, bool kFast>
__device__ __forceinline__ float* row_buffer(int e0) {
    if (kFast) return nullptr;
    __shared__ float buf[kWarps][32 * 8];
    return buf[threadIdx.x >> 5] + ((threadIdx.x & 31) / LANES) * (LANES * 8) + e0;
}

// One warp per (token, part): the heads of a token in groups of kU * 32 / LANES, the loads of
// a group issued before its arithmetic.
template <typename T, int LANES, bool kInter, bool kFast, int kU>
__device__ __forceinline__ void forward_heads(const Args& a, const T* x, int64_t hs, T* out, int H,
                                              const float* w, const Turn<LANES, kInter, kFast>& turn, int e0,
                                              int sub, int part, float* buf) {
    constexpr int kRows = 32 / LANES;  // rows a warp takes at once
    const bool live = e0 < a.D;
    float wt[8];
    const bool has_w = w != nullptr;
#pragma unroll
    for (int i = 0; i < 8; ++i) wt[i] = 1.f;
    if (has_w && live) load8(w + e0, wt);
    for (int h0 = part * kRows * kU; h0 < H; h0 += a.split * kRows * kU) {
        float v[kU][8];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int h = h0 + u * kRows + sub;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
            if (h < H && live) load8(x + h * hs + e0, v[u]);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int h = h0 + u * kRows + sub;
            if (a.norm) {
                float sq = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sq = fmaf(v[u][i], v[u][i], sq);
                const float r = norm_scale(a, row_sum<LANES>(sq));
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= r;
            }
            if (has_w) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= wt[i];
            }
            turn.template apply<false>(a, e0, v[u], buf);
            if (h < H && live) store8(out + int64_t(h) * a.D + e0, v[u]);
        }
    }
}

template <typename T, int LANES, bool kInter, bool kFast, int kU>
__global__ void __launch_bounds__(kWarps * 32) qkr_forward_kernel(const __grid_constant__ Args a) {
    const int lane = threadIdx.x & 31, e0 = (lane % LANES) * 8, sub = lane / LANES;
    const int64_t item = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t n = item / a.split;
    const int part = int(item % a.split);
    if (n >= int64_t(a.B) * a.T) return;
    const int b = int(n / a.T), t = int(n % a.T);
    float* buf = row_buffer<LANES, kFast>(e0);
    Turn<LANES, kInter, kFast> turn;
    turn.load(a, b, t, e0, lane);
    const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + t * a.qs[1];
    const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + t * a.ks[1];
    forward_heads<T, LANES, kInter, kFast, kU>(a, q, a.qs[2], static_cast<T*>(a.qo) + n * a.Hq * a.D, a.Hq, a.wq, turn, e0,
                                              sub, part, buf);
    forward_heads<T, LANES, kInter, kFast, kU>(a, k, a.ks[2], static_cast<T*>(a.ko) + n * a.Hk * a.D, a.Hk, a.wk, turn, e0,
                                              sub, part, buf);
}

// dw accumulates this thread's share of the weight gradient of its eight elements.
template <typename T, int LANES, bool kInter, bool kFast, int kU>
__device__ __forceinline__ void backward_heads(const Args& a, const T* x, int64_t hs, const T* g, T* out, int H,
                                               const float* w, const Turn<LANES, kInter, kFast>& turn, int e0,
                                               int sub, int part, float* buf, float* dw) {
    constexpr int kRows = 32 / LANES;
    const bool live = e0 < a.D;
    float wt[8];
    const bool has_w = w != nullptr;
#pragma unroll
    for (int i = 0; i < 8; ++i) wt[i] = 1.f;
    if (has_w && live) load8(w + e0, wt);
    for (int h0 = part * kRows * kU; h0 < H; h0 += a.split * kRows * kU) {
        float v[kU][8], d[kU][8];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int h = h0 + u * kRows + sub;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = d[u][i] = 0.f;
            if (h < H && live) {
                load8(g + int64_t(h) * a.D + e0, d[u]);
                if (a.norm || has_w) load8(x + h * hs + e0, v[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int h = h0 + u * kRows + sub;
            turn.template apply<true>(a, e0, d[u], buf);
            if (a.norm) {
                float sq = 0.f, ux = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sq = fmaf(v[u][i], v[u][i], sq);
                    ux = fmaf(d[u][i] * wt[i], v[u][i], ux);
                }
                sq = row_sum<LANES>(sq);
                ux = row_sum<LANES>(ux);
                const float r = norm_scale(a, sq);
                const float m = r * r * (a.norm == 1 ? ux / float(a.D) : ux);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (has_w) dw[i] = fmaf(d[u][i], v[u][i] * r, dw[i]);
                    d[u][i] = r * fmaf(-v[u][i], m, d[u][i] * wt[i]);
                }
            } else if (has_w) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dw[i] = fmaf(d[u][i], v[u][i], dw[i]);
                    d[u][i] *= wt[i];
                }
            }
            if (h < H && live) store8(out + int64_t(h) * a.D + e0, d[u]);
        }
    }
}

// A fixed grid of blocks walks the tokens, so that the weight gradients are summed in
// registers over a block's rows, then over its warps, then (qkr_weight_kernel) over the
// blocks, each in a fixed order.
template <typename T, int LANES, bool kInter, bool kFast>
__global__ void __launch_bounds__(kWarps * 32) qkr_backward_kernel(const __grid_constant__ Args a) {
    const int lane = threadIdx.x & 31, e0 = (lane % LANES) * 8, sub = lane / LANES;
    float* buf = row_buffer<LANES, kFast>(e0);
    float dwq[8], dwk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dwq[i] = dwk[i] = 0.f;
    const int64_t items = int64_t(a.B) * a.T * a.split;
    for (int64_t item = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); item < items; item += int64_t(gridDim.x) * kWarps) {
        const int64_t n = item / a.split;
        const int part = int(item % a.split), b = int(n / a.T), t = int(n % a.T);
        Turn<LANES, kInter, kFast> turn;
        turn.load(a, b, t, e0, lane);
        const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + t * a.qs[1];
        const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + t * a.ks[1];
        backward_heads<T, LANES, kInter, kFast, 2>(a, q, a.qs[2], static_cast<const T*>(a.gq) + n * a.Hq * a.D,
                                                   static_cast<T*>(a.qo) + n * a.Hq * a.D, a.Hq, a.wq, turn, e0, sub,
                                                   part, buf, dwq);
        backward_heads<T, LANES, kInter, kFast, 2>(a, k, a.ks[2], static_cast<const T*>(a.gk) + n * a.Hk * a.D,
                                                   static_cast<T*>(a.ko) + n * a.Hk * a.D, a.Hk, a.wk, turn, e0, sub,
                                                   part, buf, dwk);
    }
    if (a.part == nullptr) return;
    __shared__ float sum[kWarps][2][LANES * 8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
            dwq[i] += __shfl_xor_sync(kAll, dwq[i], o);
            dwk[i] += __shfl_xor_sync(kAll, dwk[i], o);
        }
        if (sub == 0) {
            sum[threadIdx.x >> 5][0][e0 + i] = dwq[i];
            sum[threadIdx.x >> 5][1][e0 + i] = dwk[i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.D; i += kWarps * 32) {
        const int which = i / a.D, e = i % a.D;
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x += sum[w][which][e];
        a.part[(int64_t(blockIdx.x) * 2 + which) * a.D + e] = x;
    }
}

// dw[which][e] = sum over blocks of the partials: a block per 8 elements of one weight, 32
// threads an element.
__global__ void __launch_bounds__(256) qkr_weight_kernel(const float* part, int blocks, int D, float* dwq, float* dwk) {
    const int e = blockIdx.x * 8 + (threadIdx.x & 7), which = blockIdx.y, g = threadIdx.x >> 3;
    float* out = which ? dwk : dwq;
    if (out == nullptr) return;
    float x = 0.f;
    for (int b = g; b < blocks; b += 32) x += part[(int64_t(b) * 2 + which) * D + e];
    __shared__ float sum[32][8];
    sum[g][threadIdx.x & 7] = x;
    __syncthreads();
    if (g == 0) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) y += sum[i][threadIdx.x & 7];
        out[e] = y;
    }
}

constexpr int kBackwardBlocks = 4;  // blocks a multiprocessor of the backward grid

// Warps of a token: one where the tokens alone fill the multiprocessors (the token's cos and
// sin are then read once), else as many as there are groups of heads.
int split_of(const Args& a, int lanes, int unroll) {
    const int rows = 32 / lanes;
    const int groups = (((a.Hq > a.Hk ? a.Hq : a.Hk) + rows * unroll - 1) / (rows * unroll));
    const int64_t want = int64_t(tc::sm_count()) * 32, tokens = int64_t(a.B) * a.T;
    if (tokens >= want) return 1;
    const int64_t s = (want + tokens - 1) / tokens;
    return int(s < groups ? s : groups);
}

template <typename T, int LANES, bool kInter, bool kFast, int kU>
void launch_forward(Args a, cudaStream_t s) {
    a.split = split_of(a, LANES, kU);
    const int64_t items = int64_t(a.B) * a.T * a.split;
    qkr_forward_kernel<T, LANES, kInter, kFast, kU>
        <<<unsigned((items + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a);
}

template <typename T, int LANES, bool kInter, bool kFast>
void launch(Args a, bool back, int blocks, cudaStream_t s) {
    if (back) {
        a.split = split_of(a, LANES, 2);
        qkr_backward_kernel<T, LANES, kInter, kFast><<<blocks, kWarps * 32, 0, s>>>(a);
    } else if (kFast && int64_t(a.B) * a.T >= int64_t(tc::sm_count()) * 8) {
        launch_forward<T, LANES, kInter, kFast, kFast ? 4 : 1>(a, s);
    } else {  // few tokens: one group of heads a warp
        launch_forward<T, LANES, kInter, kFast, 1>(a, s);
    }
}

template <typename T, int LANES>
void pick_layout(const Args& a, bool back, int blocks, cudaStream_t s) {
    const bool fast = a.R % (a.inter ? 8 : 16) == 0;
    if (a.inter) {
        if (fast) launch<T, LANES, true, true>(a, back, blocks, s);
        else launch<T, LANES, true, false>(a, back, blocks, s);
    } else {
        if (fast) launch<T, LANES, false, true>(a, back, blocks, s);
        else launch<T, LANES, false, false>(a, back, blocks, s);
    }
}

template <typename T>
void pick_lanes(const Args& a, bool back, int blocks, cudaStream_t s) {
    if (a.D <= 32) pick_layout<T, 4>(a, back, blocks, s);
    else if (a.D <= 64) pick_layout<T, 8>(a, back, blocks, s);
    else if (a.D <= 128) pick_layout<T, 16>(a, back, blocks, s);
    else pick_layout<T, 32>(a, back, blocks, s);
}

// blocks of the backward grid: from the sizes alone, so that the workspace can be sized on a
// host without a GPU (152 multiprocessors)
int backward_blocks(int64_t tokens) {
    const int64_t most = 152 * kBackwardBlocks, need = (tokens * 8 + kWarps - 1) / kWarps;
    return int(need < most ? need : most);
}

rm_status check(const rm_cp_qkr_problem* p, Args* a) {
    if (p == nullptr) return api_fail(RM_ERR_INVALID_ARG, "problem is null");
    if (p->B <= 0 || p->T <= 0 || p->Hq <= 0 || p->Hk <= 0 || p->D <= 0)
        return api_fail(RM_ERR_INVALID_ARG, "B, T, Hq, Hk and D must be positive");
    if (p->dtype != RM_F32 && p->dtype != RM_BF16) return api_fail(RM_ERR_INVALID_ARG, "dtype must be RM_F32 or RM_BF16");
    if (p->norm < 0 || p->norm > 2) return api_fail(RM_ERR_INVALID_ARG, "norm must be 0 (none), 1 (rms) or 2 (l2)");
    if (!(p->eps >= 0.f) || p->eps > 3.0e38f) return api_fail(RM_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (p->R < 0 || p->R > p->D || p->R % 2) return api_fail(RM_ERR_INVALID_ARG, "R must be even, in [0, D]");
    if (p->R > 0 && p->max_pos <= 0) return api_fail(RM_ERR_INVALID_ARG, "max_pos must be positive");
    if (p->pos_rows != 0 && p->pos_rows != 1 && p->pos_rows != p->B)
        return api_fail(RM_ERR_INVALID_ARG, "pos_rows must be 0 (no positions), 1 or B");
    if (p->D % 8 || p->D > 256) return api_fail(RM_ERR_UNSUPPORTED, "D must be a multiple of 8, at most 256");
    if (int64_t(p->B) * p->T > (int64_t(1) << 31) - 1) return api_fail(RM_ERR_SHAPE, "B * T exceeds 2^31 - 1");
    const int es = p->dtype == RM_F32 ? 4 : 2;
    for (int i = 0; i < 3; ++i) {
        if (p->q_stride[i] < 0 || p->k_stride[i] < 0) return api_fail(RM_ERR_INVALID_ARG, "strides must not be negative");
        if (p->q_stride[i] * es % 16 || p->k_stride[i] * es % 16)
            return api_fail(RM_ERR_ALIGNMENT, "the strides of q and k must be multiples of 16 bytes");
        a->qs[i] = p->q_stride[i];
        a->ks[i] = p->k_stride[i];
    }
    a->B = p->B, a->T = p->T, a->Hq = p->Hq, a->Hk = p->Hk, a->D = p->D, a->R = p->R, a->norm = p->norm;
    a->inter = p->interleaved ? 1 : 0, a->eps = p->eps, a->max_pos = p->max_pos, a->pos_rows = p->pos_rows;
    a->pos64 = p->pos64 ? 1 : 0;
    return RM_OK;
}

rm_status run(const rm_cp_qkr_problem* p, const Args& a, bool back, int blocks, cudaStream_t s) {
    if (p->dtype == RM_F32) pick_lanes<float>(a, back, blocks, s);
    else pick_lanes<__nv_bfloat16>(a, back, blocks, s);
    note_launch(1);
    if (!launch_ok()) {
        char msg[256];
        std::snprintf(msg, sizeof(msg), "norm and rotation launch failed: %s", cuda_error_text());
        return api_fail(RM_ERR_CUDA, msg);
    }
    return RM_OK;
}

// positions are read one at a time: aligned to their own size
rm_status check_positions(const Args& a, const void* p) {
    if (p == nullptr) return api_fail(RM_ERR_INVALID_ARG, "positions is NULL");
    if (reinterpret_cast<uintptr_t>(p) % (a.pos64 ? 8 : 4)) return api_fail(RM_ERR_ALIGNMENT, "positions is not aligned to its elements");
    return RM_OK;
}

rm_status aligned_or_null(const void* p, const char* name) { return p == nullptr ? RM_OK : api_need(p, name); }

}  // namespace
}  // namespace qkr
}  // namespace rmcp

#define RM_QKR_NEED(ptr)                            \
    do {                                            \
        rm_status s_ = rmcp::api_need((ptr), #ptr); \
        if (s_ != RM_OK) return s_;                 \
    } while (0)
#define RM_QKR_OPT(ptr)                                         \
    do {                                                        \
        rm_status s_ = rmcp::qkr::aligned_or_null((ptr), #ptr); \
        if (s_ != RM_OK) return s_;                             \
    } while (0)

extern "C" {

size_t rm_cp_qkr_workspace_size(const rm_cp_qkr_problem* p) {
    rmcp::qkr::Args a{};
    if (rmcp::qkr::check(p, &a) != RM_OK) return 0;
    return size_t(rmcp::qkr::backward_blocks(int64_t(a.B) * a.T)) * 2 * a.D * sizeof(float);
}

rm_status rm_cp_qkr_forward(const rm_cp_qkr_problem* p, const void* q, const void* k, const float* wq,
                            const float* wk, const float* table, const void* positions, void* q_out, void* k_out,
                            rm_stream_t stream) {
    rmcp::qkr::Args a{};
    rm_status st = rmcp::qkr::check(p, &a);
    if (st != RM_OK) return st;
    RM_QKR_NEED(q);
    RM_QKR_NEED(k);
    RM_QKR_NEED(q_out);
    RM_QKR_NEED(k_out);
    RM_QKR_OPT(wq);
    RM_QKR_OPT(wk);
    if (a.R > 0) RM_QKR_NEED(table);
    if (a.R > 0 && a.pos_rows > 0) {
        st = rmcp::qkr::check_positions(a, positions);
        if (st != RM_OK) return st;
    }
    a.q = q, a.k = k, a.wq = wq, a.wk = wk, a.table = table, a.qo = q_out, a.ko = k_out;
    a.pos = a.pos_rows > 0 ? positions : nullptr;
    rmcp::begin_launches();
    return rmcp::qkr::run(p, a, false, 0, reinterpret_cast<cudaStream_t>(stream));
}

rm_status rm_cp_qkr_backward(const rm_cp_qkr_problem* p, const void* q, const void* k, const float* wq,
                             const float* wk, const float* table, const void* positions, const void* dq_out,
                             const void* dk_out, void* dq, void* dk, float* dwq, float* dwk, void* ws,
                             rm_stream_t stream) {
    rmcp::qkr::Args a{};
    rm_status st = rmcp::qkr::check(p, &a);
    if (st != RM_OK) return st;
    RM_QKR_NEED(q);
    RM_QKR_NEED(k);
    RM_QKR_NEED(dq_out);
    RM_QKR_NEED(dk_out);
    RM_QKR_NEED(dq);
    RM_QKR_NEED(dk);
    RM_QKR_OPT(wq);
    RM_QKR_OPT(wk);
    RM_QKR_OPT(dwq);
    RM_QKR_OPT(dwk);
    if (a.R > 0) RM_QKR_NEED(table);
    if (a.R > 0 && a.pos_rows > 0) {
        st = rmcp::qkr::check_positions(a, positions);
        if (st != RM_OK) return st;
    }
    if ((dwq != nullptr && wq == nullptr) || (dwk != nullptr && wk == nullptr))
        return rmcp::api_fail(RM_ERR_INVALID_ARG, "a weight's gradient needs the weight");
    const bool weights = dwq != nullptr || dwk != nullptr;
    if (weights) RM_QKR_NEED(ws);
    a.q = q, a.k = k, a.wq = wq, a.wk = wk, a.table = table, a.gq = dq_out, a.gk = dk_out, a.qo = dq, a.ko = dk;
    a.pos = a.pos_rows > 0 ? positions : nullptr;
    a.part = weights ? static_cast<float*>(ws) : nullptr;
    const int blocks = rmcp::qkr::backward_blocks(int64_t(a.B) * a.T);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    rmcp::begin_launches();
    st = rmcp::qkr::run(p, a, true, blocks, s);
    if (st != RM_OK || !weights) return st;
    rmcp::qkr::qkr_weight_kernel<<<dim3(a.D / 8, 2), 256, 0, s>>>(a.part, blocks, a.D, dwq, dwk);
    rmcp::note_launch(1);
    if (!rmcp::launch_ok()) return rmcp::api_fail(RM_ERR_CUDA, "weight gradient launch failed");
    return RM_OK;
}

}  // extern "C"
