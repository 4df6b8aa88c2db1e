// rms_kernels.cu -- root-mean-square norm of rows, with the residual's addition before it, a gate, and an
// output in 8 bits with scales (rm_cp_rms_*), forward and backward.
//
// Per row x in R^n, with residual q, gate z and weight w (each optional), a(z) = z / (1 + e^-z):
//     h = x + q (rounded to the residual's type and kept),   u = h  or  h a(z)  (gate first)
//     y = u r w  or  u r w a(z),   r = (sum u^2 / n + eps)^(-1/2)
// In 8 bits: s = max |y| of a group of elements / 448 (at least 2^-126), y8 = e4m3(y / s).
// Backward, with e = dy a(z) (gate after) or dy, d = e w:
//     du = r (d - u r (r sum d u / n)),   dw = sum over rows of e u r
//     dz = dy u r w a'(z),  or du h a'(z) (gate first);   dh = du [a(z)] + what comes down the residual stream
//
// Bound by HBM: a row stays in registers between its sums and its outputs, so that every input is read and
// every output written once.  Sums and the arithmetic are fp32; an output is rounded once.  In bf16, us in a CUDA graph: 32768
// rows of 2048 with a residual 85 (6.3 TB/s), their backward 92 (5.8); 32768 x 16 gated rows of 128 69 (5.8), their backward 114
// (5.9); 8191 rows of 4096 in 8 bits 53 (4.5: two thirds of the issue slots go into the conversions).
#include <cuda_fp8.h>

#include <cstdio>
#include <type_traits>

#include "internal.h"
#include "pairs.cuh"
#include "tc_tiles.cuh"

namespace rmcp {
namespace rms {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kTiny = 1.17549435e-38f;  // 2^-126: the smallest scale
constexpr float kF8Max = 448.f;

struct Args {
    int N, H, n;
    float eps, inv_n;
    int group;                    // elements of a scale; 0: the row
    int64_t xs[2], rs[2], zs[2];  // token and head strides (elements) of x, of the residual (backward: h), of the gate
    const void* x;                // backward: dy
    const void* res;              // backward: h
    const void* z;
    const float* w;
    const void* dh;               // backward: the gradient of h from the residual stream
    void* h;                      // backward: dresidual, where its type is not that of dx
    void* y;                      // or y8; backward: dx
    void* dz;
    float* scale;
    float* part;                  // backward: [blocks][n] partial weight gradients
};

// Eight elements
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) { tc::unpack8(*reinterpret_cast<const uint4*>(p), x); }
__device__ __forceinline__ void store8(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) { *reinterpret_cast<uint4*>(p) = tc::pack8(x); }

// What is kept of a gate's sigmoid s.  fp32: that of -|z|, the smaller of s and 1 - s, so that both are off by 7 u at most (u
// = 2^-24: 2 of the exponential, 1 of the sum, 4 of the quotient) whatever z is.  bf16: s itself by the quick functions, off by
// some (8 + |z|) u, far below bf16's 2^-8.  (16384 x 16 rows of 128 in fp32: 8 bits 54 us, with bf16's functions 47 and with a
// quotient to nearest 62; fp32 outputs and the backward are bound by HBM all the same.)
template <typename T>
__device__ __forceinline__ float squash(float z) {
    if constexpr (sizeof(T) == 4) {
        const float e = expf(-fabsf(z));
        return __fdividef(e, 1.f + e);
    } else {
        return __fdividef(1.f, 1.f + __expf(-z));
    }
}
template <typename T>
__device__ __forceinline__ float sigmoid(float z, float kept) { return sizeof(T) == 4 && z >= 0.f ? 1.f - kept : kept; }
template <typename T>
__device__ __forceinline__ float one_less_sigmoid(float z, float kept) { return sizeof(T) == 4 && z >= 0.f ? kept : 1.f - kept; }
template <typename T>
__device__ __forceinline__ float silu(float z) { return z * sigmoid<T>(z, squash<T>(z)); }

// Eight elements as they lie in memory
template <typename T>
struct Raw {
    uint4 x[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < int(sizeof(T)) / 2; ++i) x[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < int(sizeof(T)) / 2; ++i) x[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float* y) const {
        if constexpr (sizeof(T) == 2) tc::unpack8(x[0], y);
        else load8(reinterpret_cast<const float*>(x), y);
    }
    __device__ __forceinline__ void pairs(uint64_t* y) const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) y[i] = widen2(w[i]);
            else y[i] = pair(w[2 * i], w[2 * i + 1]);
        }
    }
    // pairs rounded to T
    __device__ __forceinline__ void set(const uint64_t* y) {
        uint32_t* w = reinterpret_cast<uint32_t*>(x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) w[i] = pack2(y[i]);
            else unpair(y[i], w[2 * i], w[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < int(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = x[i];
    }
};
__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }

// Threads of a row: LANES of a warp (several rows a warp), or with LANES 0 the whole block.
// Sums x and y over them; the largest of the bits m.  (The bits of |y| order as the values do, with NaN above all.)
template <int LANES, typename M>
__device__ __forceinline__ void row_reduce(float& x, M& m, int& turn) {
    auto join = [](M p, M q) { return std::is_same<M, float>::value ? M(p + q) : (p > q ? p : q); };
#pragma unroll
    for (int o = (LANES ? LANES : 32) / 2; o > 0; o >>= 1) {
        x += __shfl_xor_sync(kAll, x, o);
        m = join(m, __shfl_xor_sync(kAll, m, o));
    }
    if constexpr (LANES == 0) {
        __shared__ float xs[2][32];
        __shared__ M ms[2][32];
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) xs[turn][threadIdx.x >> 5] = x, ms[turn][threadIdx.x >> 5] = m;
        __syncthreads();
        x = lane < warps ? xs[turn][lane] : 0.f, m = lane < warps ? ms[turn][lane] : M(0);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            x += __shfl_xor_sync(kAll, x, o);
            m = join(m, __shfl_xor_sync(kAll, m, o));
        }
        turn ^= 1;  // (the next row's sums go elsewhere: a slow warp may still read these)
    }
}

// This thread's row of those that a block takes at once, its place in the row, and the threads of a row
template <int LANES>
__device__ __forceinline__ int row_of_block() { return LANES ? int(threadIdx.x) / (LANES ? LANES : 1) : 0; }
template <int LANES>
__device__ __forceinline__ int place_in_row() { return LANES ? int(threadIdx.x) % (LANES ? LANES : 1) : int(threadIdx.x); }
template <int LANES>
__device__ __forceinline__ int row_threads() { return LANES ? LANES : int(blockDim.x); }
__device__ __forceinline__ void place(const Args& a, int64_t row, int& t, int& h) {
    t = a.H == 1 ? int(row) : int(uint32_t(row) / uint32_t(a.H));
    h = int(row - int64_t(t) * a.H);
}

// What a thread reads of a row
template <typename T, typename R, bool kRes, bool kGate, int VPT>
struct Row {
    Raw<T> x[VPT], z[kGate ? VPT : 1];
    Raw<R> q[kRes ? VPT : 1];
};

// A thread has VPT times eight elements of a row: those of unit i are 8 (place + i threads) ..  A block goes on to the
// rows gridDim.x further on, whose loads are under way while it takes a row.
// kGate: 0 none, 1 after the norm, 2 before it.
template <typename T, typename R, bool kRes, int kGate, bool kQuant, int LANES, int VPT, int TPB>
__global__ void __launch_bounds__(TPB) rms_forward_kernel(const __grid_constant__ Args a) {
    constexpr bool kAhead = VPT == 1;
    const int RPB = LANES ? TPB / (LANES ? LANES : 1) : 1, at = place_in_row<LANES>(), step = row_threads<LANES>();
    const int64_t rows = int64_t(a.N) * a.H, hop = int64_t(gridDim.x) * RPB;
    int64_t row = int64_t(blockIdx.x) * RPB + row_of_block<LANES>();
    int turn = 0;
    Row<T, R, kRes, kGate != 0, VPT> next;
    auto load = [&](int64_t r) {
        int t, hd;
        place(a, r < rows ? r : 0, t, hd);
        const T* x = static_cast<const T*>(a.x) + t * a.xs[0] + hd * a.xs[1];
        const R* q = kRes ? static_cast<const R*>(a.res) + t * a.rs[0] + hd * a.rs[1] : nullptr;
        const T* z = kGate ? static_cast<const T*>(a.z) + t * a.zs[0] + hd * a.zs[1] : nullptr;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int e = 8 * (at + i * step);
            const bool live = r < rows && e < a.n;
            if (live) next.x[i].load(x + e);
            else next.x[i].zero();
            if (kRes) {
                if (live) next.q[i].load(q + e);
                else next.q[i].zero();
            }
            if (kGate) {
                if (live) next.z[i].load(z + e);
                else next.z[i].zero();
            }
        }
    };
    load(row);
    for (int64_t first = int64_t(blockIdx.x) * RPB; first < rows; first += hop, row += hop) {
        const Row<T, R, kRes, kGate != 0, VPT> now = next;
        if (kAhead && first + hop < rows) load(row + hop);
        const bool there = row < rows;
        uint64_t m[VPT][4], squares = 0;  // pairs of elements
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int e = 8 * (at + i * step);
            const bool live = there && e < a.n;
            uint64_t b[4], act[4];
            now.x[i].pairs(m[i]);
            if (kRes) {
                now.q[i].pairs(b);
#pragma unroll
                for (int j = 0; j < 4; ++j) m[i][j] = add2(m[i][j], b[j]);
                Raw<R> h;
                h.set(m[i]);
                if (live) h.store(static_cast<R*>(a.h) + row * a.n + e);
                h.pairs(m[i]);
            }
            if (kGate) {
                float z[8];
                now.z[i].get(z);
#pragma unroll
                for (int j = 0; j < 4; ++j) act[j] = pair(silu<T>(z[2 * j]), silu<T>(z[2 * j + 1]));
            }
            if (kGate == 2) {
#pragma unroll
                for (int j = 0; j < 4; ++j) m[i][j] = mul2(m[i][j], act[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) squares = fma2(m[i][j], m[i][j], squares);
            if (a.w != nullptr && live) {
                Raw<float> w;
                w.load(a.w + e);
                w.pairs(b);
#pragma unroll
                for (int j = 0; j < 4; ++j) m[i][j] = mul2(m[i][j], b[j]);
            }
            if (kGate == 1) {
#pragma unroll
                for (int j = 0; j < 4; ++j) m[i][j] = mul2(m[i][j], act[j]);
            }
        }
        uint32_t lo, hi;
        unpair(squares, lo, hi);
        float sq = __uint_as_float(lo) + __uint_as_float(hi);
        uint32_t big[VPT], most = 0;
        if (kQuant) {
            // (a NaN in the row is in its sum, and so in r and every scale)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    unpair(m[i][j], lo, hi);
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(lo)), fabsf(__uint_as_float(hi))));
                }
                big[i] = __float_as_uint(top);
                most = max(most, big[i]);
            }
        }
        row_reduce<LANES>(sq, most, turn);
        const float r = rsqrtf(fmaf(sq, a.inv_n, a.eps));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int e = 8 * (at + i * step);
            const bool live = there && e < a.n;
            if (kQuant) {
                uint32_t top = most;
                if (a.group) {
                    top = big[i];
                    for (int o = a.group / 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
                }
                // (the scale is off by three roundings, its inverse by two ulps more: in y8, far below e4m3's 2^-4)
                float s = __uint_as_float(top) * r * (1.f / kF8Max);
                s = s < kTiny ? kTiny : s;  // (a NaN stays)
                const float f = __fdividef(1.f, s);  // (r f may leave fp32 where y is all but 0)
                uint32_t out[2];
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    uint32_t p[4];
                    unpair(mul2(mul2(m[i][j], both(r)), both(f)), p[0], p[1]);
                    unpair(mul2(mul2(m[i][j + 1], both(r)), both(f)), p[2], p[3]);
                    const __nv_fp8x2_storage_t x = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(p[0]), __uint_as_float(p[1])), __NV_SATFINITE, __NV_E4M3);
                    const __nv_fp8x2_storage_t y = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(p[2]), __uint_as_float(p[3])), __NV_SATFINITE, __NV_E4M3);
                    out[j / 2] = uint32_t(x) | uint32_t(y) << 16;
                }
                if (live) {
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + row * a.n + e) = make_uint2(out[0], out[1]);
                    const int of = a.group ? a.group : a.n;
                    if (e % of == 0) a.scale[row * (a.n / of) + e / of] = s;
                }
            } else if (live) {
#pragma unroll
                for (int j = 0; j < 4; ++j) m[i][j] = mul2(m[i][j], both(r));
                Raw<T> y;
                y.set(m[i]);
                y.store(static_cast<T*>(a.y) + row * a.n + e);
            }
        }
        if (!kAhead && first + hop < rows) load(row + hop);
    }
}

// Threads of a multiprocessor that a backward is compiled for: as many as its registers allow (fp32 with a gate, 16384 x 16 rows of
// 128: 104 us at 128 registers; at 80, with spills, 187, gate first 216)
template <typename T, typename R, int kGate>
constexpr int backward_threads() { return kGate && sizeof(T) == 4 ? 512 : kGate || sizeof(T) == 4 || sizeof(R) == 4 ? 768 : 1024; }

// Rows are taken in a fixed order by a fixed number of blocks, so that the weight's gradient does not depend on the
// launch.  With one unit a thread a row's inputs, dh among them, are on their way while the row before is taken, and the weights
// stay in registers.  What was read stays as it was read (bf16: half the registers) between the sums and the outputs.
template <typename T, typename R, int kGate, bool kDh, bool kTwo, int LANES, int VPT, int TPB>
__global__ void __launch_bounds__(TPB, VPT > 1 || TPB > backward_threads<T, R, kGate>() ? 1 : backward_threads<T, R, kGate>() / TPB) rms_backward_kernel(const __grid_constant__ Args a) {
    constexpr bool kAhead = VPT == 1;
    const int RPB = LANES ? TPB / (LANES ? LANES : 1) : 1, at = place_in_row<LANES>(), step = row_threads<LANES>();
    const int64_t rows = int64_t(a.N) * a.H, hop = int64_t(gridDim.x) * RPB;
    int64_t row = int64_t(blockIdx.x) * RPB + row_of_block<LANES>();
    int turn = 0;
    float ws[8], dw[VPT][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        ws[j] = 1.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) dw[i][j] = 0.f;
    }
    if (kAhead && a.w != nullptr && 8 * at < a.n) load8(a.w + 8 * at, ws);
    struct In {
        Raw<R> h[VPT], dh[kDh ? VPT : 1];
        Raw<T> d[VPT], z[kGate ? VPT : 1];
    } next;
    auto load = [&](int64_t r) {
        int t, hd;
        place(a, r < rows ? r : 0, t, hd);
        const R* h = static_cast<const R*>(a.res) + t * a.rs[0] + hd * a.rs[1];
        const T* z = kGate ? static_cast<const T*>(a.z) + t * a.zs[0] + hd * a.zs[1] : nullptr;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int e = 8 * (at + i * step);
            if (r < rows && e < a.n) {
                next.h[i].load(h + e);
                next.d[i].load(static_cast<const T*>(a.x) + r * a.n + e);
                if (kGate) next.z[i].load(z + e);
                if (kDh) next.dh[i].load(static_cast<const R*>(a.dh) + r * a.n + e);
            } else {
                next.h[i].zero(), next.d[i].zero();
                if (kGate) next.z[i].zero();
            }
        }
    };
    load(row);
    for (int64_t first = int64_t(blockIdx.x) * RPB; first < rows; first += hop, row += hop) {
        const In now = next;
        if (kAhead && first + hop < rows) load(row + hop);
        float sg[kGate ? VPT : 1][8], sq = 0.f, du = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float u[8], d[8], zz[8], wl[8];
            now.h[i].get(u);
            now.d[i].get(d);
            if (kGate) now.z[i].get(zz);
            if (!kAhead && a.w != nullptr && 8 * (at + i * step) < a.n) load8(a.w + 8 * (at + i * step), wl);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (kGate) sg[i][j] = squash<T>(zz[j]);
                const float act = kGate ? zz[j] * sigmoid<T>(zz[j], sg[i][j]) : 1.f, w = kAhead ? ws[j] : a.w != nullptr ? wl[j] : 1.f;
                const float uu = kGate == 2 ? u[j] * act : u[j];
                const float dd = (kGate == 1 ? d[j] * act : d[j]) * w;
                sq = fmaf(uu, uu, sq);
                if (8 * (at + i * step) < a.n) du = fmaf(dd, uu, du);
            }
        }
        row_reduce<LANES>(sq, du, turn);
        const float r = rsqrtf(fmaf(sq, a.inv_n, a.eps)), c = r * du * a.inv_n;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int e = 8 * (at + i * step);
            if (row < rows && e < a.n) {
                float u[8], d[8], zz[8], wl[8], add[8], dz[8], out[8];
                now.h[i].get(u);
                now.d[i].get(d);
                if (kGate) now.z[i].get(zz);
                if (kDh) now.dh[i].get(add);
                if (!kAhead && a.w != nullptr) load8(a.w + e, wl);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float s = kGate ? sigmoid<T>(zz[j], sg[i][j]) : 0.f, w = kAhead ? ws[j] : a.w != nullptr ? wl[j] : 1.f;
                    const float act = kGate ? zz[j] * s : 1.f, slope = kGate ? s * fmaf(zz[j], one_less_sigmoid<T>(zz[j], sg[i][j]), 1.f) : 0.f;
                    const float uh = (kGate == 2 ? u[j] * act : u[j]) * r;
                    const float ee = kGate == 1 ? d[j] * act : d[j];
                    dw[i][j] = fmaf(ee, uh, dw[i][j]);
                    float g = r * fmaf(ee, w, -uh * c);
                    if (kGate == 1) dz[j] = d[j] * uh * w * slope;
                    if (kGate == 2) dz[j] = g * u[j] * slope, g *= act;
                    out[j] = kDh ? g + add[j] : g;
                }
                if (kGate) store8(static_cast<T*>(a.dz) + row * a.n + e, dz);
                if (kTwo) store8(static_cast<R*>(a.h) + row * a.n + e, out);
                store8(static_cast<T*>(a.y) + row * a.n + e, out);
            }
        }
        if (!kAhead && first + hop < rows) load(row + hop);
    }
    if (a.part == nullptr) return;
    float* to = a.part + int64_t(blockIdx.x) * a.n;
    if constexpr (LANES > 0) {  // the block's rows, group after group
        __shared__ float sum[LANES * VPT * 8];
        for (int g = 0; g < RPB; ++g) {
            if (row_of_block<LANES>() == g) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float& s = sum[8 * (at + i * step) + j];
                        s = g ? s + dw[i][j] : dw[i][j];
                    }
            }
            __syncthreads();
        }
        for (int e = threadIdx.x; e < a.n; e += TPB) to[e] = sum[e];
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int e = 8 * (at + i * step);
            if (e < a.n) store8(to + e, dw[i]);
        }
    }
}

// dw[e] = sum of the blocks' parts: 32 columns a block, 32 threads a column
__global__ void __launch_bounds__(1024) rms_weight_kernel(const float* part, float* dw, int blocks, int n) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    float x = 0.f;
    if (e < n) {
#pragma unroll 4
        for (int b = g; b < blocks; b += 32) x += part[int64_t(b) * n + e];
    }
    s[g][lane] = x;
    __syncthreads();
    x = warp_sum(s[lane][g]);
    if (lane == 0 && blockIdx.x * 32 + g < n) dw[blockIdx.x * 32 + g] = x;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// f(LANES, VPT, TPB) of the row length and the direction.  Rows of up to 256 elements take the lanes of a warp, longer ones a block of as
// many warps as they need, with eight elements a thread: more of them in a thread leave fewer loads under way (16384 rows of
// 4096: 85 us, and with two units of eight a thread 92).
template <bool kBackward, typename F>
auto by_length(int n, F f) {
    using std::integral_constant;
#define RM_RMS_SHAPE(l, v, t) f(integral_constant<int, l>{}, integral_constant<int, v>{}, integral_constant<int, t>{})
    if (n <= 64) return RM_RMS_SHAPE(8, 1, 256);
    if (n <= 128) return RM_RMS_SHAPE(16, 1, 256);
    if (n <= 256) return RM_RMS_SHAPE(32, 1, 256);
    if (n <= 1024) return RM_RMS_SHAPE(0, 1, 128);
    if (n <= 2048) return RM_RMS_SHAPE(0, 1, 256);
    if (n <= 4096) return RM_RMS_SHAPE(0, 1, 512);
    if constexpr (!kBackward)
        if (n <= 8192) return RM_RMS_SHAPE(0, 1, 1024);
    if (n <= 8192) return RM_RMS_SHAPE(0, 2, 512);
    if (n <= 16384) return RM_RMS_SHAPE(0, 2, 1024);
    return RM_RMS_SHAPE(0, 4, 1024);
#undef RM_RMS_SHAPE
}
int threads_of(int n, int LANES, int VPT, int TPB) {
    const int need = ((n + 8 * VPT - 1) / (8 * VPT) + 31) / 32 * 32;
    return LANES ? TPB : need < TPB ? need : TPB;
}
int blocks_of(int64_t rows, int LANES, int TPB, int64_t most) {
    const int64_t per = LANES ? TPB / LANES : 1, b = (rows + per - 1) / per;
    return int(b < most ? b : most);
}

// Blocks of a backward, whose partial gradients the workspace holds: as many as run at once
int blocks_of_backward(int n, int threads = 1024) {
    return by_length<true>(n, [&](auto l, auto v, auto t) {
        const int each = (v() > 1 ? t() : threads) / threads_of(n, l, v, t);
        return 152 * (each > 0 ? each : 1);
    });
}

rm_status launched() {
    note_launch(1);
    if (launch_ok()) return RM_OK;
    char msg[256];
    std::snprintf(msg, sizeof(msg), "norm: launch failed: %s", cuda_error_text());
    return api_fail(RM_ERR_CUDA, msg);
}

template <typename T, typename R, bool kRes, int kGate>
rm_status forward(const Args& a, cudaStream_t s) {
    const int64_t rows = int64_t(a.N) * a.H;
    return by_length<false>(a.n, [&](auto l, auto v, auto t) {
        // With a gate, whose arithmetic would leave the memory idle, and for long rows, blocks go on to further rows whose
        // loads are ahead (gated, 32768 x 16 rows of 128: 69 us, a block for its rows alone 80; rows of 4096: 85 and 109);
        // else a block has its rows alone (32768 rows of 2048: 85 us, and 89 with 2048 threads a multiprocessor going on)
        const int threads = threads_of(a.n, l, v, t), blocks = blocks_of(rows, l, t, kGate || a.n > 2048 ? 152 * (1024 / threads) : 0x7fffffff);
        if (a.scale != nullptr) rms_forward_kernel<T, R, kRes, kGate, true, l(), v(), t()><<<blocks, threads, 0, s>>>(a);
        else rms_forward_kernel<T, R, kRes, kGate, false, l(), v(), t()><<<blocks, threads, 0, s>>>(a);
        return launched();
    });
}

template <typename T, typename R, int kGate, bool kDh, bool kTwo>
rm_status backward(const Args& a, float* dw, cudaStream_t s) {
    const int64_t rows = int64_t(a.N) * a.H;
    return by_length<true>(a.n, [&](auto l, auto v, auto t) {
        const int threads = threads_of(a.n, l, v, t), blocks = blocks_of(rows, l, t, blocks_of_backward(a.n, backward_threads<T, R, kGate>()));
        rms_backward_kernel<T, R, kGate, kDh, kTwo, l(), v(), t()><<<blocks, threads, 0, s>>>(a);
        const rm_status st = launched();
        if (st != RM_OK || dw == nullptr) return st;
        rms_weight_kernel<<<(a.n + 31) / 32, 1024, 0, s>>>(a.part, dw, blocks, a.n);
        return launched();
    });
}

struct Shape {
    bool bf16, res_bf16;
    int gate;
};

rm_status check(const rm_cp_rms_problem* p, Args* a, Shape* k) {
    if (p == nullptr) return api_fail(RM_ERR_INVALID_ARG, "problem is null");
    if (p->N < 0 || p->H <= 0 || p->n <= 0) return api_fail(RM_ERR_INVALID_ARG, "H and n must be positive, N not negative");
    if ((p->dtype != RM_F32 && p->dtype != RM_BF16) || (p->res_dtype != RM_F32 && p->res_dtype != RM_BF16))
        return api_fail(RM_ERR_INVALID_ARG, "dtype and res_dtype must be RM_F32 or RM_BF16");
    if (p->dtype == RM_F32 && p->res_dtype != RM_F32) return api_fail(RM_ERR_UNSUPPORTED, "fp32 rows need an fp32 residual");
    if (!(p->eps >= 0.f && p->eps < 3.0e38f)) return api_fail(RM_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (p->gate < 0 || p->gate > 2) return api_fail(RM_ERR_INVALID_ARG, "gate must be 0, 1 or 2");
    if (p->n % 8 || p->n > 32768) return api_fail(RM_ERR_UNSUPPORTED, "n must be a multiple of 8 up to 32768");
    if (p->group != 0 && (p->group != 32 && p->group != 64 && p->group != 128)) return api_fail(RM_ERR_UNSUPPORTED, "group must be 0, 32, 64 or 128");
    if (p->group && p->n % p->group) return api_fail(RM_ERR_SHAPE, "group must divide n");
    if (int64_t(p->N) * p->H > (int64_t(1) << 31) - 1) return api_fail(RM_ERR_SHAPE, "too many rows");
    const int es = p->dtype == RM_F32 ? 4 : 2, rs = p->res_dtype == RM_F32 ? 4 : 2;
    for (int i = 0; i < 2; ++i) {
        if (p->x_stride[i] < 0 || p->r_stride[i] < 0 || p->z_stride[i] < 0) return api_fail(RM_ERR_INVALID_ARG, "strides must not be negative");
        if (p->x_stride[i] * es % 16 || p->r_stride[i] * rs % 16 || p->z_stride[i] * es % 16)
            return api_fail(RM_ERR_ALIGNMENT, "strides must be multiples of 16 bytes");
        a->xs[i] = p->x_stride[i], a->rs[i] = p->r_stride[i], a->zs[i] = p->z_stride[i];
    }
    a->N = p->N, a->H = p->H, a->n = p->n, a->eps = p->eps, a->inv_n = 1.f / float(p->n);
    a->group = p->group == p->n ? 0 : p->group;
    *k = Shape{p->dtype == RM_BF16, p->res_dtype == RM_BF16, p->gate};
    return RM_OK;
}

template <typename T, typename R, bool kRes>
rm_status forward_gates(const Args& a, const Shape& k, cudaStream_t s) {
    return k.gate == 0 ? forward<T, R, kRes, 0>(a, s) : k.gate == 1 ? forward<T, R, kRes, 1>(a, s) : forward<T, R, kRes, 2>(a, s);
}
rm_status forward_any(const Args& a, const Shape& k, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (a.res == nullptr) return k.bf16 ? forward_gates<B, B, false>(a, k, s) : forward_gates<float, float, false>(a, k, s);
    if (!k.bf16) return forward<float, float, true, 0>(a, s);
    return k.res_bf16 ? forward<B, B, true, 0>(a, s) : forward<B, float, true, 0>(a, s);
}

template <typename T, typename R, int kGate>
rm_status backward_dh(const Args& a, float* dw, cudaStream_t s) {
    constexpr bool kTwo = !std::is_same<T, R>::value;
    if (kGate) return backward<T, R, kGate, false, kTwo>(a, dw, s);
    return a.dh ? backward<T, R, 0, true, kTwo>(a, dw, s) : backward<T, R, 0, false, kTwo>(a, dw, s);
}
rm_status backward_any(const Args& a, const Shape& k, float* dw, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (k.bf16 && !k.res_bf16) return backward_dh<B, float, 0>(a, dw, s);
    if (k.bf16) return k.gate == 0 ? backward_dh<B, B, 0>(a, dw, s) : k.gate == 1 ? backward_dh<B, B, 1>(a, dw, s) : backward_dh<B, B, 2>(a, dw, s);
    return k.gate == 0   ? backward_dh<float, float, 0>(a, dw, s)
           : k.gate == 1 ? backward_dh<float, float, 1>(a, dw, s)
                         : backward_dh<float, float, 2>(a, dw, s);
}

rm_status aligned(const void* p, const char* name, int size) {
    if (p != nullptr && reinterpret_cast<uintptr_t>(p) % size == 0) return RM_OK;
    char msg[96];
    std::snprintf(msg, sizeof(msg), "%s is %s", name, p ? "not aligned" : "NULL");
    return api_fail(p ? RM_ERR_ALIGNMENT : RM_ERR_INVALID_ARG, msg);
}

// Bytes that a tensor [N,H,n] with the given strides reaches over
int64_t reach(const rm_cp_rms_problem* p, const int64_t* st, int es) { return ((p->N - 1) * st[0] + (p->H - 1) * st[1] + p->n) * es; }

struct Range {
    const void* at;
    int64_t bytes;
    bool dense;  // contiguous: an output of the same size may lie exactly on it
};
// Whether an output meets another tensor otherwise than by being one it may replace
bool meets(const Range& out, const Range& other, bool may_replace) {
    if (out.at == nullptr || other.at == nullptr || out.bytes <= 0 || other.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(out.at), y = reinterpret_cast<uintptr_t>(other.at);
    if (x + uint64_t(out.bytes) <= y || y + uint64_t(other.bytes) <= x) return false;
    return !(may_replace && x == y && out.bytes == other.bytes && other.dense);
}
bool dense(const rm_cp_rms_problem* p, const int64_t* st) {
    return (p->H == 1 || st[1] == p->n) && (p->N <= 1 || st[0] == int64_t(p->H) * p->n);
}

}  // namespace
}  // namespace rms
}  // namespace rmcp

#define RM_RMS_NEED(ptr, size)                                        \
    do {                                                              \
        rm_status s_ = rmcp::rms::aligned((ptr), #ptr, (size));       \
        if (s_ != RM_OK) return s_;                                   \
    } while (0)

extern "C" {

static rm_status rms_forward(const rm_cp_rms_problem* p, const void* x, const void* residual, const void* gate, const float* weight,
                             void* h, void* y, float* scales, bool quant, rm_stream_t stream) {
    using namespace rmcp;
    rms::Args a{};
    rms::Shape k;
    rm_status st = rms::check(p, &a, &k);
    if (st != RM_OK) return st;
    if (residual != nullptr && k.gate) return api_fail(RM_ERR_UNSUPPORTED, "a residual and a gate exclude one another");
    if (p->N == 0) return RM_OK;
    RM_RMS_NEED(x, 16);
    if (residual != nullptr) {
        RM_RMS_NEED(residual, 16);
        RM_RMS_NEED(h, 16);
    }
    if (k.gate) RM_RMS_NEED(gate, 16);
    if (weight != nullptr) RM_RMS_NEED(weight, 16);
    RM_RMS_NEED(y, 16);
    if (quant) RM_RMS_NEED(scales, 4);
    const int es = k.bf16 ? 2 : 4, rs = k.res_bf16 ? 2 : 4;
    const int64_t all = int64_t(p->N) * p->H * p->n;
    const rms::Range rx{x, rms::reach(p, p->x_stride, es), rms::dense(p, p->x_stride)}, rw{weight, int64_t(p->n) * 4, false},
        rr{residual, rms::reach(p, p->r_stride, rs), rms::dense(p, p->r_stride)}, rz{k.gate ? gate : nullptr, rms::reach(p, p->z_stride, es), rms::dense(p, p->z_stride)},
        ry{y, all * (quant ? 1 : es), true}, rh{residual ? h : nullptr, all * rs, true},
        rsc{quant ? scales : nullptr, int64_t(p->N) * p->H * (a.group ? p->n / a.group : 1) * 4, true};
    const bool bad = rms::meets(ry, rx, !quant) || rms::meets(ry, rr, false) || rms::meets(ry, rz, false) || rms::meets(ry, rw, false) ||
                     rms::meets(rh, rx, false) || rms::meets(rh, rr, true) || rms::meets(rh, rw, false) || rms::meets(rh, ry, false) ||
                     rms::meets(rsc, rx, false) || rms::meets(rsc, rr, false) || rms::meets(rsc, rz, false) || rms::meets(rsc, rw, false) ||
                     rms::meets(rsc, ry, false) || rms::meets(rsc, rh, false);
    if (bad) return api_fail(RM_ERR_INVALID_ARG, "an output overlaps another tensor (only h may replace the residual, and y replace x)");
    a.x = x, a.res = residual, a.z = gate, a.w = weight, a.h = h, a.y = y, a.scale = quant ? scales : nullptr;
    begin_launches();
    return rms::forward_any(a, k, reinterpret_cast<cudaStream_t>(stream));
}

rm_status rm_cp_rms_forward(const rm_cp_rms_problem* p, const void* x, const void* residual, const void* gate, const float* weight,
                            void* h, void* y, rm_stream_t stream) {
    return rms_forward(p, x, residual, gate, weight, h, y, nullptr, false, stream);
}

rm_status rm_cp_rms_quant(const rm_cp_rms_problem* p, const void* x, const void* residual, const void* gate, const float* weight,
                          void* h, void* y8, float* scales, rm_stream_t stream) {
    return rms_forward(p, x, residual, gate, weight, h, y8, scales, true, stream);
}

size_t rm_cp_rms_workspace_size(const rm_cp_rms_problem* p) {
    rmcp::rms::Args a{};
    rmcp::rms::Shape k;
    if (rmcp::rms::check(p, &a, &k) != RM_OK) return 0;
    return size_t(rmcp::rms::blocks_of_backward(a.n)) * size_t(a.n) * sizeof(float);
}

rm_status rm_cp_rms_backward(const rm_cp_rms_problem* p, const void* h, const void* gate, const float* weight, const void* dy,
                             const void* dh, void* dx, void* dresidual, void* dgate, float* dweight, void* ws, rm_stream_t stream) {
    using namespace rmcp;
    rms::Args a{};
    rms::Shape k;
    rm_status st = rms::check(p, &a, &k);
    if (st != RM_OK) return st;
    const bool two = k.bf16 && !k.res_bf16;
    if ((dh != nullptr || two) && k.gate) return api_fail(RM_ERR_UNSUPPORTED, "a residual and a gate exclude one another");
    if (dweight != nullptr && weight == nullptr) return api_fail(RM_ERR_INVALID_ARG, "the weight's gradient without the weight");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (p->N == 0) {  // no rows: their sum is 0
        if (dweight == nullptr) return RM_OK;
        RM_RMS_NEED(dweight, 4);
        begin_launches();
        rms::rms_weight_kernel<<<(a.n + 31) / 32, 1024, 0, s>>>(nullptr, dweight, 0, a.n);
        return rms::launched();
    }
    RM_RMS_NEED(h, 16);
    RM_RMS_NEED(dy, 16);
    RM_RMS_NEED(dx, 16);
    if (k.gate) {
        RM_RMS_NEED(gate, 16);
        RM_RMS_NEED(dgate, 16);
    }
    if (weight != nullptr) RM_RMS_NEED(weight, 16);
    if (dh != nullptr) RM_RMS_NEED(dh, 16);
    if (two) RM_RMS_NEED(dresidual, 16);
    if (dweight != nullptr) {
        RM_RMS_NEED(dweight, 4);
        RM_RMS_NEED(ws, 16);
    }
    const int es = k.bf16 ? 2 : 4, rs = k.res_bf16 ? 2 : 4;
    const int64_t all = int64_t(p->N) * p->H * p->n;
    const rms::Range in[] = {{h, rms::reach(p, p->r_stride, rs), rms::dense(p, p->r_stride)}, {dy, all * es, true}, {dh, all * rs, true},
                             {k.gate ? gate : nullptr, rms::reach(p, p->z_stride, es), rms::dense(p, p->z_stride)}},
                     out[] = {{dx, all * es, true}, {two ? dresidual : nullptr, all * rs, true}, {k.gate ? dgate : nullptr, all * es, true},
                              {dweight, int64_t(p->n) * 4, false}, {dweight ? ws : nullptr, int64_t(rms::blocks_of_backward(p->n)) * p->n * 4, false}},
                     w{weight, int64_t(p->n) * 4, false};
    bool bad = false;
    for (int i = 0; i < 5; ++i) {
        for (const rms::Range& x : in) bad |= rms::meets(out[i], x, i < 3);
        for (int j = 0; j < i; ++j) bad |= rms::meets(out[i], out[j], false);
        bad |= rms::meets(out[i], w, false);
    }
    if (bad) return api_fail(RM_ERR_INVALID_ARG, "an output overlaps another tensor");
    a.x = dy, a.res = h, a.z = gate, a.w = weight, a.dh = dh, a.h = dresidual, a.y = dx, a.dz = dgate;
    a.part = dweight ? static_cast<float*>(ws) : nullptr;
    begin_launches();
    return rms::backward_any(a, k, dweight, s);
}

}  // extern "C"
