// clip_kernels.cu -- the global norm of many tensors and the scaling that clips them
// (rm_cp_clip_grad_norm).
//     norm = sqrt(sum_i sum g_i^2),   out_i = g_i min(1, max_norm / (norm + eps))
//
// Bound by HBM: the norm reads every gradient, the scaling reads it again and writes it.  The
// tensors are cut into pieces of kPiece elements; a fixed grid of blocks walks the pieces of
// up to kMany tensors whose addresses and sizes travel in the launch's parameters, so that no
// table is copied to the device first.  The scaling walks the pieces from the last one, so
// that what the norm read last is still in L2.  Each block adds up its pieces, every block of
// the scaling adds up the blocks' sums in one order, and no atomics are used: the result
// depends on the sizes alone.
//
// 311 tensors of 805 million elements, two thirds of them bf16: 1.07 ms, of which the norm 330 us at 6.4 TB/s;
// the second read makes the floor 938 us.  Pieces of 16384 elements on four blocks a multiprocessor took
// 1.23 ms.  75 small tensors of 2 million elements: 25 us on the device, 11 of them the norm (with pieces of this
// size they are on some 120 of the 912 blocks), and the host's path of 75 us, most of it collecting addresses.
#include <algorithm>
#include <cstdio>
#include <new>
#include <vector>

#include "tc_tiles.cuh"

namespace rmcp {
namespace clip {

using tc::pack8;
using tc::unpack8;

namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 32768;   // elements: 128 a thread
constexpr int kBlocks = 152 * 6;
// Tensors of a launch: few are passed in a small block of parameters (75 tensors: 3 us less on the device and
// 8 less on the host than in the large one), many in as large a block as there is.
constexpr int kFew = 96, kMany = 900;

template <int N>
struct Batch {
    const void* in[N];
    void* out[N];
    int64_t numel[N];
    int64_t first[N + 1];       // first piece of each tensor
    uint8_t in_bf16[N], out_bf16[N];
    int n;
};
static_assert(sizeof(Batch<kMany>) + 64 <= 32764, "the parameters of a launch");

// Tensor of piece p.
template <int N>
__device__ __forceinline__ int find(const Batch<N>& b, int64_t p) {
    int lo = 0, hi = b.n - 1;  // first[lo] <= p < first[hi + 1]
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.first[mid] <= p) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float load1(const float* p) { return __ldcs(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* x) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
    unpack8(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) { *reinterpret_cast<uint4*>(p) = pack8(x); }

// elements before the first 16-byte boundary of p, at most n
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
    const int h = int(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
    return h < n ? h : n;
}

// This thread's share of one piece: sum of squares and largest magnitude (NaN does not count
// in the latter; it is in the sum).
template <typename T>
__device__ __forceinline__ void square_piece(const T* p, int n, float* sum, float* most) {
    float s = 0.f, m = 0.f;
    const int head = head_of(p, n), body = (n - head) / 8, tail = head + body * 8;
    if (int(threadIdx.x) < head) {
        const float x = load1(p + threadIdx.x);
        s = x * x, m = fabsf(x);
    }
    const T* q = p + head;
#pragma unroll 4
    for (int i = threadIdx.x; i < body; i += kThreads) {
        float x[8];
        load8(q + i * 8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s = fmaf(x[e], x[e], s);
            m = fmaxf(m, fabsf(x[e]));
        }
    }
    if (tail + int(threadIdx.x) < n) {
        const float x = load1(p + tail + threadIdx.x);
        s = fmaf(x, x, s), m = fmaxf(m, fabsf(x));
    }
    *sum = s, *most = m;
}
template <typename T>
__device__ __noinline__ double square_piece_wide(const T* p, int n) {
    double s = 0.;
    const int head = head_of(p, n), body = (n - head) / 8, tail = head + body * 8;
    if (int(threadIdx.x) < head) {
        const double x = load1(p + threadIdx.x);
        s += x * x;
    }
    for (int i = threadIdx.x; i < body; i += kThreads)
        for (int e = 0; e < 8; ++e) {
            const double x = load1(p + head + i * 8 + e);
            s += x * x;
        }
    if (tail + int(threadIdx.x) < n) {
        const double x = load1(p + tail + threadIdx.x);
        s += x * x;
    }
    return s;
}

// A thread's share of a piece is at most 130 elements.  Its squares stay inside fp32 when the
// largest magnitude is in [1e-15, 1e18]: above, they could overflow; below, the squares
// (< 1e-30) could lose bits to fp32's smallest numbers (1.2e-38), so they are summed in fp64.
__device__ __forceinline__ bool in_range(float m) { return m == 0.f || (m >= 1e-15f && m <= 1e18f); }

__device__ __forceinline__ double block_sum(double x) {
    __shared__ double sum[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0) sum[threadIdx.x >> 5] = x;
    __syncthreads();
    double y = 0.;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) y += sum[w];
    __syncthreads();
    return y;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 6) clip_square_kernel(const __grid_constant__ Batch<N> b, double* part) {
    double total = 0.;
    for (int64_t p = blockIdx.x; p < b.first[b.n]; p += gridDim.x) {
        const int t = find(b, p);
        const int64_t at = (p - b.first[t]) * kPiece, left = b.numel[t] - at;
        const int n = left < kPiece ? int(left) : kPiece;
        float s, m;
        if (b.in_bf16[t]) {
            const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(b.in[t]) + at;
            square_piece(x, n, &s, &m);
            total += in_range(m) ? double(s) : square_piece_wide(x, n);
        } else {
            const float* x = static_cast<const float*>(b.in[t]) + at;
            square_piece(x, n, &s, &m);
            total += in_range(m) ? double(s) : square_piece_wide(x, n);
        }
    }
    const double y = block_sum(total);
    if (threadIdx.x == 0) part[blockIdx.x] = y;
}

// The norm from the blocks' sums; every block of a launch comes to the same value.
__device__ __forceinline__ double norm_of(const double* part, int n) {
    double x = 0.;
    for (int i = threadIdx.x; i < n; i += kThreads) x += part[i];
    return sqrt(block_sum(x));
}

__global__ void __launch_bounds__(kThreads) clip_norm_kernel(const double* part, int n, float* norm) {
    const double x = norm_of(part, n);
    if (threadIdx.x == 0) *norm = float(x);
}

template <typename TI, typename TO>
__device__ __forceinline__ void scale_piece(const TI* p, TO* o, int n, float c) {
    // 16-byte accesses on both sides where one head brings both to a boundary
    const int head = head_of(p, n);
    if (head == n || (reinterpret_cast<uintptr_t>(o + head) & 15) == 0) {
        const int body = (n - head) / 8, tail = head + body * 8;
        if (int(threadIdx.x) < head) o[threadIdx.x] = from_f32<TO>(load1(p + threadIdx.x) * c);
        const TI* q = p + head;
        TO* r = o + head;
#pragma unroll 4
        for (int i = threadIdx.x; i < body; i += kThreads) {
            float x[8];
            load8(q + i * 8, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= c;
            store8(r + i * 8, x);
        }
        if (tail + int(threadIdx.x) < n) o[tail + threadIdx.x] = from_f32<TO>(load1(p + tail + threadIdx.x) * c);
    } else {
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += kThreads) o[i] = from_f32<TO>(load1(p + i) * c);
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 6)
    clip_scale_kernel(const __grid_constant__ Batch<N> b, const double* part, int parts, float max_norm, float eps, float* norm) {
    const double x = norm_of(part, parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = float(x);
    // fminf would drop a NaN: the comparison keeps it
    const double f = double(max_norm) / (x + double(eps));
    const float c = f > 1. ? 1.f : float(f);
    const int64_t pieces = b.first[b.n];
    for (int64_t i = blockIdx.x; i < pieces; i += gridDim.x) {
        const int64_t p = pieces - 1 - i;
        const int t = find(b, p);
        const int64_t at = (p - b.first[t]) * kPiece, left = b.numel[t] - at;
        const int n = left < kPiece ? int(left) : kPiece;
        const int how = b.in_bf16[t] * 2 + b.out_bf16[t];
        const float* pf = static_cast<const float*>(b.in[t]) + at;
        const __nv_bfloat16* ph = static_cast<const __nv_bfloat16*>(b.in[t]) + at;
        float* of = static_cast<float*>(b.out[t]) + at;
        __nv_bfloat16* oh = static_cast<__nv_bfloat16*>(b.out[t]) + at;
        if (how == 3) scale_piece(ph, oh, n, c);
        else if (how == 2) scale_piece(ph, of, n, c);
        else if (how == 1) scale_piece(pf, oh, n, c);
        else scale_piece(pf, of, n, c);
    }
}

struct Call {
    int n;
    const void* const* grads;
    const int64_t* numels;
    const int32_t* dtypes;
    void* const* outs;
    const int32_t* out_dtypes;
};

// Whether an output lies over another output or over a gradient that is not its own: blocks read and write them in
// no order.  (Memory in ascending order, as the parts of one buffer are, is not sorted.)
bool overlapping(const Call& c) {
    struct Range {
        uintptr_t begin, end;
        bool out;
    };
    std::vector<Range> r;
    r.reserve(2 * size_t(c.n));
    for (int i = 0; i < c.n; ++i) {
        if (c.numels[i] == 0) continue;
        const uintptr_t g = reinterpret_cast<uintptr_t>(c.grads[i]), o = reinterpret_cast<uintptr_t>(c.outs[i]);
        if (g != o) r.push_back({g, g + uintptr_t(c.numels[i]) * (c.dtypes[i] == RM_F32 ? 4 : 2), false});
        r.push_back({o, o + uintptr_t(c.numels[i]) * (c.out_dtypes[i] == RM_F32 ? 4 : 2), true});
    }
    auto before = [](const Range& x, const Range& y) { return x.begin < y.begin; };
    if (!std::is_sorted(r.begin(), r.end(), before)) std::sort(r.begin(), r.end(), before);
    uintptr_t any = 0, out = 0;  // ends of what was passed
    for (const Range& x : r) {
        if (x.begin < (x.out ? any : out)) return true;
        any = std::max(any, x.end);
        if (x.out) out = std::max(out, x.end);
    }
    return false;
}

// Tensors [t0, t0 + N) of the call.
template <int N>
void fill(const Call& c, int t0, Batch<N>* b) {
    b->n = c.n - t0 < N ? c.n - t0 : N;
    int64_t at = 0;
    for (int i = 0; i < b->n; ++i) {
        const int t = t0 + i;
        b->in[i] = c.grads[t];
        b->out[i] = c.outs ? c.outs[t] : nullptr;
        b->numel[i] = c.numels[t];
        b->in_bf16[i] = c.dtypes[t] == RM_BF16;
        b->out_bf16[i] = c.outs && c.out_dtypes[t] == RM_BF16;
        b->first[i] = at;
        at += (c.numels[t] + kPiece - 1) / kPiece;
    }
    b->first[b->n] = at;
}

template <int N>
bool run(const Call& c, float max_norm, float eps, float* norm, double* part, cudaStream_t s) {
    Batch<N> b;
    const int batches = (c.n + N - 1) / N;
    for (int i = 0; i < batches; ++i) {
        fill(c, i * N, &b);
        clip_square_kernel<N><<<kBlocks, kThreads, 0, s>>>(b, part + int64_t(i) * kBlocks);
        note_launch(1);
        if (!launch_ok()) return false;
    }
    if (c.outs == nullptr) {
        clip_norm_kernel<<<1, kThreads, 0, s>>>(part, batches * kBlocks, norm);
        note_launch(1);
        return launch_ok();
    }
    for (int i = batches - 1; i >= 0; --i) {
        if (batches > 1) fill(c, i * N, &b);
        clip_scale_kernel<N><<<kBlocks, kThreads, 0, s>>>(b, part, batches * kBlocks, max_norm, eps, norm);
        note_launch(1);
        if (!launch_ok()) return false;
    }
    return true;
}

}  // namespace
}  // namespace clip
}  // namespace rmcp

extern "C" {

size_t rm_cp_clip_workspace_size(int32_t n) {
    if (n <= 0) return 0;
    return size_t((n + rmcp::clip::kMany - 1) / rmcp::clip::kMany) * rmcp::clip::kBlocks * sizeof(double);
}

rm_status rm_cp_clip_grad_norm(int32_t n, const void* const* grads, const int64_t* numels, const int32_t* dtypes,
                               void* const* outs, const int32_t* out_dtypes, float max_norm, float eps, float* norm,
                               void* ws, rm_stream_t stream) {
    using rmcp::api_fail;
    if (n <= 0) return api_fail(RM_ERR_INVALID_ARG, "n must be positive");
    if (grads == nullptr || numels == nullptr || dtypes == nullptr) return api_fail(RM_ERR_INVALID_ARG, "grads, numels and dtypes must not be NULL");
    if (outs != nullptr && out_dtypes == nullptr) return api_fail(RM_ERR_INVALID_ARG, "out_dtypes must not be NULL with outs");
    if (outs != nullptr && !(max_norm >= 0.f && max_norm <= 3.4e38f)) return api_fail(RM_ERR_INVALID_ARG, "max_norm must be finite and not negative");
    if (!(eps >= 0.f && eps <= 3.4e38f)) return api_fail(RM_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (norm == nullptr || reinterpret_cast<uintptr_t>(norm) % 4) return api_fail(norm ? RM_ERR_ALIGNMENT : RM_ERR_INVALID_ARG, "norm is NULL or not aligned");
    rm_status st = rmcp::api_need(ws, "ws");
    if (st != RM_OK) return st;
    for (int i = 0; i < n; ++i) {
        if (numels[i] < 0) return api_fail(RM_ERR_INVALID_ARG, "a tensor has a negative size");
        if (numels[i] > (int64_t(1) << 46)) return api_fail(RM_ERR_SHAPE, "a tensor is too large");
        for (int side = 0; side < (outs ? 2 : 1); ++side) {
            const int32_t dt = side ? out_dtypes[i] : dtypes[i];
            if (dt != RM_F32 && dt != RM_BF16) return api_fail(RM_ERR_INVALID_ARG, "dtypes must be RM_F32 or RM_BF16");
            const void* p = side ? outs[i] : grads[i];
            if (numels[i] == 0) continue;
            if (p == nullptr) return api_fail(RM_ERR_INVALID_ARG, "a tensor's pointer is NULL");
            if (side && p == grads[i] && dt != dtypes[i]) return api_fail(RM_ERR_INVALID_ARG, "in place, a tensor keeps its dtype");
            if (reinterpret_cast<uintptr_t>(p) % (dt == RM_F32 ? 4 : 2)) return api_fail(RM_ERR_ALIGNMENT, "a tensor is not aligned to its elements");
        }
    }
    const rmcp::clip::Call c{n, grads, numels, dtypes, outs, out_dtypes};
    try {
        if (outs != nullptr && rmcp::clip::overlapping(c)) return api_fail(RM_ERR_INVALID_ARG, "an output overlaps another output or another gradient");
    } catch (const std::bad_alloc&) {
        return api_fail(RM_ERR_INVALID_ARG, "out of host memory");
    }
    rmcp::begin_launches();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool ok = n <= rmcp::clip::kFew ? rmcp::clip::run<rmcp::clip::kFew>(c, max_norm, eps, norm, static_cast<double*>(ws), s)
                                          : rmcp::clip::run<rmcp::clip::kMany>(c, max_norm, eps, norm, static_cast<double*>(ws), s);
    if (ok) return RM_OK;
    char msg[256];
    std::snprintf(msg, sizeof(msg), "gradient norm launch failed: %s", rmcp::cuda_error_text());
    return api_fail(RM_ERR_CUDA, msg);
}

}  // extern "C"
