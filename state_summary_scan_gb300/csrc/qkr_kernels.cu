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
// keeps one token's cos and sin in registers over that token's heads.  Long inputs go through
// qkr_stream_kernel.  32768 tokens, 16 + 16 heads of 128 in bf16: forward 95 us (5.7 TB/s), backward with
// both weight gradients 136 us (5.9 TB/s); one token of 32 + 8 heads: 2.9 us, a launch.  (All times here: calls
// one after another in a CUDA graph, on inputs that together exceed the L2.)
#include <cstdio>

#include "pairs.cuh"
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

// Eight fp32 values as pairs.
__device__ __forceinline__ void load_pairs(const float* p, uint64_t* x) {
    const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2*>(p)), b = __ldg(reinterpret_cast<const ulonglong2*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }
__device__ __forceinline__ uint64_t swapped(uint64_t p) {
    uint32_t x, y;
    unpair(p, x, y);
    return pair(y, x);
}

// Eight elements as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint32_t x[4];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    }
    __device__ __forceinline__ void shared(const __nv_bfloat16* p) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    }
    __device__ __forceinline__ void zero() { x[0] = x[1] = x[2] = x[3] = 0; }
    __device__ __forceinline__ void pairs(uint64_t* v) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pair(x[i] << 16, x[i] & 0xffff0000u);
    }
    __device__ __forceinline__ Raw from(int lane) const {
        Raw r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.x[i] = __shfl_sync(kAll, x[i], lane);
        return r;
    }
};
template <>
struct Raw<float> {
    uint64_t x[4];
    __device__ __forceinline__ void load(const float* p) { load_pairs(p, x); }
    __device__ __forceinline__ void shared(const float* p) {
        const ulonglong2 a = reinterpret_cast<const ulonglong2*>(p)[0], b = reinterpret_cast<const ulonglong2*>(p)[1];
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    }
    __device__ __forceinline__ void zero() { x[0] = x[1] = x[2] = x[3] = 0; }
    __device__ __forceinline__ void pairs(uint64_t* v) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = x[i];
    }
    __device__ __forceinline__ Raw from(int lane) const {
        Raw r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t u, v;
            unpair(x[i], u, v);
            r.x[i] = pair(__shfl_sync(kAll, u, lane), __shfl_sync(kAll, v, lane));
        }
        return r;
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const uint64_t* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u, v;
        unpair(x[i], u, v);
        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(u), __uint_as_float(v));
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const uint64_t* x) {
    reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(x[0], x[1]);
    reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(x[2], x[3]);
}

// Sum of a lane's eight products over the LANES lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(uint64_t p) {
    uint32_t u, v;
    unpair(p, u, v);
    float x = __uint_as_float(u) + __uint_as_float(v);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}

// Row and token of token n of B * T (below 2^31).
__device__ __forceinline__ void place(const Args& a, int64_t n, int& b, int& t) {
    b = int(uint32_t(n) / uint32_t(a.T));
    t = int(uint32_t(n) - uint32_t(b) * uint32_t(a.T));
}

// Position of token t of row b; -1 where it lies outside the table.
__device__ __forceinline__ int position(const Args& a, int b, int t) {
    if (a.R == 0) return 0;
    if (a.pos == nullptr) return t < a.max_pos ? t : -1;
    const int64_t i = (a.pos_rows > 1 ? int64_t(b) * a.T : 0) + t;
    const int64_t p = a.pos64 ? __ldg(static_cast<const long long*>(a.pos) + i)
                              : int64_t(__ldg(static_cast<const int*>(a.pos) + i));
    return p >= 0 && p < a.max_pos ? int(p) : -1;
}

// The rotation of a lane's eight elements e0 .. e0 + 7, of which those below R turn: element e
// becomes x_e c_e + x_p s_e, with p the other member of its pair and s_e negative for the first of a
// pair; the transposed rotation has -s_e.  Elements that do not turn have c = 1, s = 0.
// kFast: R is a multiple of 16 (half layout) or 8 (interleaved), so a lane's elements turn together
// and their partners sit in one lane (from) or in the lane itself; otherwise each element finds its
// own partner through the warp's row buffer.
template <typename T, int LANES, bool kInter, bool kFast>
struct Turn {
    uint64_t c[4], s[4];
    bool on;
    int from;

    __device__ __forceinline__ void load(const Args& a, int p, int e0, int lane) {
        load(a, a.table + int64_t(p < 0 ? 0 : p) * a.R, p < 0, e0, lane);
    }
    // row: the position's row of the table, in global or shared memory; bad: outside the table
    __device__ __forceinline__ void load(const Args& a, const float* row, bool bad, int e0, int lane) {
        from = lane;
        on = e0 < a.R;
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = both(1.f), s[i] = 0;
        if (!on) return;
        const int h = a.R / 2;
        const float nan = __int_as_float(0x7fffffff);
        if (kFast && kInter) {
            uint64_t x[2], y[2];
            const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(row + e0 / 2), v = *reinterpret_cast<const ulonglong2*>(row + h + e0 / 2);
            x[0] = u.x, x[1] = u.y, y[0] = v.x, y[1] = v.y;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t c0, c1, s0, s1;
                unpair(x[i / 2], c0, c1);
                unpair(y[i / 2], s0, s1);
                const float cc = __uint_as_float(i & 1 ? c1 : c0), ss = __uint_as_float(i & 1 ? s1 : s0);
                c[i] = both(bad ? nan : cc);  // (a position outside the table: NaN)
                s[i] = pair(-ss, ss);
            }
        } else if (kFast) {
            const bool first = e0 < h;
            const int at = first ? e0 : e0 - h;
            const ulonglong2* x = reinterpret_cast<const ulonglong2*>(row + at);
            const ulonglong2* y = reinterpret_cast<const ulonglong2*>(row + h + at);
            c[0] = x[0].x, c[1] = x[0].y, c[2] = x[1].x, c[3] = x[1].y;
            s[0] = y[0].x, s[1] = y[0].y, s[2] = y[1].x, s[3] = y[1].y;
            from = first ? lane + h / 8 : lane - h / 8;
            const uint64_t sign = both(first ? -1.f : 1.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i] = mul2(s[i], sign);
                if (bad) c[i] = both(nan);
            }
        } else {
            float cc[8], ss[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i;
                cc[i] = 1.f, ss[i] = 0.f;
                if (e >= a.R) continue;
                const int at = kInter ? e / 2 : (e < h ? e : e - h);
                const bool first = kInter ? !(e & 1) : e < h;
                cc[i] = bad ? nan : row[at];
                ss[i] = first ? -row[h + at] : row[h + at];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = pair(cc[2 * i], cc[2 * i + 1]), s[i] = pair(ss[2 * i], ss[2 * i + 1]);
        }
    }

    __device__ __forceinline__ void transpose() {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = mul2(s[i], both(-1.f));
    }

    // The partners of a lane's elements x (v: as pairs), 0 for those that do not turn.  Whole-warp call.
    __device__ __forceinline__ void partners(const Args& a, const Raw<T>& x, const uint64_t* v, int e0, float* buf, uint64_t* o) const {
        if (kFast && kInter) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = swapped(v[i]);
        } else if (kFast) {
            x.from(from).pairs(o);
        } else {
            const int h = a.R / 2;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t u, w;
                unpair(v[i], u, w);
                buf[2 * i] = __uint_as_float(u), buf[2 * i + 1] = __uint_as_float(w);
            }
            __syncwarp();
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i, p = kInter ? (e ^ 1) : (e < h ? e + h : e - h);
                y[i] = e < a.R ? buf[p - e0] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = pair(y[2 * i], y[2 * i + 1]);
        }
        if (kFast && a.R < a.D && !on) o[0] = o[1] = o[2] = o[3] = 0;
    }
    // The element that a lane's element i is paired with, for its weight; itself where it does not turn.
    __device__ __forceinline__ int partner(const Args& a, int e) const {
        const int h = a.R / 2;
        return e >= a.R ? e : kInter ? (e ^ 1) : (e < h ? e + h : e - h);
    }
};

// r of a row, from its sum of squares (inv: 1 / D for rms, 1 for l2).  Without eps r reaches 1e22, and r^2 leaves
// fp32: the backward takes r (r sum u x).
__device__ __forceinline__ float norm_scale(const Args& a, float sq, float inv) { return rsqrtf(fmaf(sq, inv, a.eps)); }
__device__ __forceinline__ float mean_factor(const Args& a) { return a.norm == 1 ? 1.f / float(a.D) : 1.f; }

template <int LANES, bool kFast>
__device__ __forceinline__ float* row_buffer(int e0) {
    if (kFast) return nullptr;
    __shared__ float buf[kWarps][32 * 8];
    return buf[threadIdx.x >> 5] + ((threadIdx.x & 31) / LANES) * (LANES * 8) + e0;
}

// A warp takes 32 / LANES tokens side by side, LANES lanes each, and their heads in groups of kU,
// those of q and then those of k: every split-th group.  (Rows of one token side by side instead
// leave lanes idle where the heads are few: one head of 64 over 123,000 tokens took 251 us that way.)
// The next group's loads are issued before this group's arithmetic, and the first ones of a token
// before its cos and sin, which wait for its position.
template <int LANES, int kU>
struct Groups {
    static constexpr int kTokens = 32 / LANES;
    int nq, n;  // groups of q, and all
    __device__ __forceinline__ explicit Groups(const Args& a) : nq((a.Hq + kU - 1) / kU), n(nq + (a.Hk + kU - 1) / kU) {}
    __device__ __forceinline__ bool of_q(int g) const { return g < nq; }
    __device__ __forceinline__ int head(int g) const { return (g < nq ? g : g - nq) * kU; }
};

// Row of head h of x: of the input, with its strides, or of a contiguous [B * T, H, D].
template <typename T>
__device__ __forceinline__ const T* row_in(const Args& a, bool q, int b, int t, int h) {
    return q ? static_cast<const T*>(a.q) + b * a.qs[0] + t * a.qs[1] + h * a.qs[2]
             : static_cast<const T*>(a.k) + b * a.ks[0] + t * a.ks[1] + h * a.ks[2];
}
__device__ __forceinline__ int64_t row_at(const Args& a, bool q, int64_t n, int h) { return (n * (q ? a.Hq : a.Hk) + h) * a.D; }

// the weights of a lane's elements (1 without weights)
__device__ __forceinline__ void weights(const float* w, bool live, int e0, uint64_t* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = both(1.f);
    if (w != nullptr && live) load_pairs(w + e0, x);
}

// The weights go into the factors of the rotation, once a token and tensor, and the norm's scale
// onto the result:  y_e = r (x_e (w_e c_e) + x_p (w_p s_e)).
template <typename T, int LANES, bool kInter, bool kFast, int kU>
__global__ void __launch_bounds__(kWarps * 32, 3) qkr_forward_kernel(const __grid_constant__ Args a) {
    const int lane = threadIdx.x & 31, e0 = (lane % LANES) * 8, sub = lane / LANES;
    const Groups<LANES, kU> groups(a);
    constexpr int kTokens = Groups<LANES, kU>::kTokens;
    // (tokens * split: a split is taken where the tokens are few, so the items fit 32 bits)
    const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5), set = item / uint32_t(a.split);
    const int64_t first = int64_t(set) * kTokens, tokens = int64_t(a.B) * a.T, n = first + sub;
    if (first >= tokens) return;
    const bool live = e0 < a.D && n < tokens;
    int b, t;
    place(a, n < tokens ? n : first, b, t);
    float* buf = row_buffer<LANES, kFast>(e0);
    const int p = position(a, b, t);
    const float inv = mean_factor(a);
    auto fetch = [&](int g, Raw<T>* x) {
        const bool q = groups.of_q(g);
        const int h0 = groups.head(g), left = (q ? a.Hq : a.Hk) - h0;
        const int64_t hs = q ? a.qs[2] : a.ks[2];
        const T* from = row_in<T>(a, q, b, t, h0) + e0;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            x[u].zero();
            if (live && u < left) x[u].load(from + u * hs);
        }
    };
    Raw<T> x[kU];
    int g = int(item - set * uint32_t(a.split));
    if (g < groups.n) fetch(g, x);
    for (int side = 0; side < 2; ++side) {  // q's groups, then k's
        const bool q = side == 0;
        const int end = q ? groups.nq : groups.n;
        if (g >= end) continue;
        const float* wt = q ? a.wq : a.wk;
        Turn<T, LANES, kInter, kFast> turn;
        turn.load(a, p, e0, lane);
        if (wt != nullptr && live) {
            uint64_t w[4];
            load_pairs(wt + e0, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                turn.c[i] = mul2(turn.c[i], w[i]);
                turn.s[i] = mul2(turn.s[i], pair(__ldg(wt + turn.partner(a, e0 + 2 * i)), __ldg(wt + turn.partner(a, e0 + 2 * i + 1))));
            }
        }
        T* out = static_cast<T*>(q ? a.qo : a.ko);
        for (; g < end; g += a.split) {
            Raw<T> ahead[kU];
            if (g + a.split < groups.n) fetch(g + a.split, ahead);
            const int h0 = groups.head(g), left = (q ? a.Hq : a.Hk) - h0;
            T* to = out + row_at(a, q, n, h0) + e0;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                uint64_t v[4], o[4];
                x[u].pairs(v);
                turn.partners(a, x[u], v, e0, buf, o);
                uint64_t r = both(1.f);
                if (a.norm) {
                    uint64_t sq = mul2(v[0], v[0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) sq = fma2(v[i], v[i], sq);
                    r = both(norm_scale(a, row_sum<LANES>(sq), inv));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = mul2(r, fma2(o[i], turn.s[i], mul2(v[i], turn.c[i])));
                if (live && u < left) store8(to + u * a.D, v);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) x[u] = ahead[u];
        }
    }
}

// A fixed grid of blocks walks the tokens, so that the weight gradients are summed in registers over
// a block's rows, then over its warps, then (qkr_weight_kernel) over the blocks, each in a fixed order.
template <typename T, int LANES, bool kInter, bool kFast>
__global__ void __launch_bounds__(kWarps * 32, 2) qkr_backward_kernel(const __grid_constant__ Args a) {
    constexpr int kU = 2;
    const int lane = threadIdx.x & 31, e0 = (lane % LANES) * 8, sub = lane / LANES;
    float* buf = row_buffer<LANES, kFast>(e0);
    const Groups<LANES, kU> groups(a);
    constexpr int kTokens = Groups<LANES, kU>::kTokens;
    uint64_t dw[2][4];  // of q's and k's weights
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[0][i] = dw[1][i] = 0;
    const float inv = mean_factor(a);
    const int64_t tokens = int64_t(a.B) * a.T;
    // a warp keeps its part of every step-th set of tokens; warps that are left over have none
    const int warp = blockIdx.x * kWarps + (threadIdx.x >> 5), part = warp % a.split;
    const int64_t step = int64_t(gridDim.x * kWarps / a.split) * kTokens;
    int64_t first = warp < int(gridDim.x) * kWarps / a.split * a.split ? int64_t(warp / a.split) * kTokens : tokens, n = 0;
    int b = 0, t = 0;
    bool live = false;
    auto begin = [&]() {  // this lane's token of the set
        n = first + sub;
        live = e0 < a.D && n < tokens;
        place(a, n < tokens ? n : first, b, t);
    };
    auto fetch = [&](int g, Raw<T>* x, Raw<T>* d) {
        const bool q = groups.of_q(g);
        const int h0 = groups.head(g), left = (q ? a.Hq : a.Hk) - h0;
        const int64_t hs = q ? a.qs[2] : a.ks[2];
        const T* from = row_in<T>(a, q, b, t, h0) + e0;
        const T* grad = static_cast<const T*>(q ? a.gq : a.gk) + row_at(a, q, n, h0) + e0;
        const bool need = a.norm || (q ? a.wq : a.wk) != nullptr;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            x[u].zero();
            d[u].zero();
            if (live && u < left) {
                d[u].load(grad + u * a.D);
                if (need) x[u].load(from + u * hs);
            }
        }
    };
    if (first < tokens && part < groups.n) {
        Raw<T> x[kU], dy[kU];
        begin();
        int p = position(a, b, t), g = part;
        fetch(g, x, dy);
        uint64_t w[4];
        while (true) {
            Turn<T, LANES, kInter, kFast> turn;
            turn.load(a, p, e0, lane);
            turn.transpose();
            const int64_t n0 = n;
            const bool live0 = live;
            bool more = true;
#pragma unroll
            for (int side = 0; side < 2; ++side) {  // q's groups, then k's
                const bool q = side == 0;
                const int end = q ? groups.nq : groups.n;
                if (g >= end) continue;
                weights(q ? a.wq : a.wk, e0 < a.D, e0, w);
                T* out = static_cast<T*>(q ? a.qo : a.ko);
                while (g < end) {
                    // the group after this one: of this token, or the first of the warp's next token
                    const int g0 = g;
                    Raw<T> ax[kU], ad[kU];
                    g += a.split;
                    if (g >= groups.n) {
                        first += step;
                        more = first < tokens;
                        if (more) {
                            begin();
                            p = position(a, b, t);
                            fetch(part, ax, ad);
                        }
                    } else {
                        fetch(g, ax, ad);
                    }
                    const int h0 = groups.head(g0), left = (q ? a.Hq : a.Hk) - h0;
                    T* to = out + row_at(a, q, n0, h0) + e0;
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        uint64_t v[4], d[4], o[4];
                        x[u].pairs(v);
                        dy[u].pairs(d);
                        turn.partners(a, dy[u], d, e0, buf, o);
#pragma unroll
                        for (int i = 0; i < 4; ++i) d[i] = fma2(o[i], turn.s[i], mul2(d[i], turn.c[i]));
                        uint64_t dv[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) dv[i] = mul2(d[i], v[i]), d[i] = mul2(d[i], w[i]);
                        uint64_t r2 = both(1.f);
                        if (a.norm) {
                            uint64_t sq = mul2(v[0], v[0]), ux = mul2(dv[0], w[0]);
#pragma unroll
                            for (int i = 1; i < 4; ++i) sq = fma2(v[i], v[i], sq), ux = fma2(dv[i], w[i], ux);
                            // (a row that is not there adds 0 to the weights' gradients: its own r is infinite without eps)
                            const float ss = row_sum<LANES>(sq), r = live0 && u < left ? norm_scale(a, ss, inv) : 0.f, m = r * (r * row_sum<LANES>(ux)) * inv;
                            r2 = both(r);
                            const uint64_t m2 = both(-m);
#pragma unroll
                            for (int i = 0; i < 4; ++i) d[i] = mul2(r2, fma2(v[i], m2, d[i]));
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) dw[side][i] = fma2(dv[i], r2, dw[side][i]);
                        if (live0 && u < left) store8(to + u * a.D, d);
                    }
#pragma unroll
                    for (int u = 0; u < kU; ++u) x[u] = ax[u], dy[u] = ad[u];
                }
            }
            if (!more) break;
            g = part;
        }
    }
    float dwq[8], dwk[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u, v;
        unpair(dw[0][i], u, v);
        dwq[2 * i] = __uint_as_float(u), dwq[2 * i + 1] = __uint_as_float(v);
        unpair(dw[1][i], u, v);
        dwk[2 * i] = __uint_as_float(u), dwk[2 * i + 1] = __uint_as_float(v);
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

// ---------------------------------------------------------------------------
// The same with the rows brought in by bulk copies: each warp owns two stages of shared memory and
// fills one with the next item (all of q's or of k's heads of a token, their gradients, and the
// token's row of the table) while it works on the other.  The loop above waits for memory between
// its groups; this one needs a token's heads side by side in memory, and enough of them to be worth
// a copy.  us, the loop / this kernel, forward and backward:
//     16 + 16 heads of 128, bf16, 8192 tokens     34 / 28      56 / 45
//     the same, 32768 tokens                      101 / 95     172 / 136
//     8 + 4 heads of 128, bf16, 32768 tokens      48 / 48      77 / 68
//     16 + 16 heads of 64, fp32, 32768 tokens     96 / 98      148 / 133
// Three blocks of eight warps forward, one of twelve backward: the stages fill the shared memory.
// ---------------------------------------------------------------------------
template <bool kBack>
struct Stream {
    static constexpr int kWarps = kBack ? 12 : 8;      // of a block
    static constexpr int kBlocks = kBack ? 1 : 3;      // blocks a multiprocessor
    static constexpr uint32_t kMost = 222 * 1024 / (kWarps * kBlocks * 2) / 128 * 128;  // bytes of a stage
    static uint32_t stage(const Args& a, int es) {
        return uint32_t((a.Hq > a.Hk ? a.Hq : a.Hk) * a.D * es * (kBack ? 2 : 1) + a.R * 4);
    }
};

template <typename T, int LANES, bool kInter, bool kBack>
__global__ void __launch_bounds__(Stream<kBack>::kWarps * 32, Stream<kBack>::kBlocks) qkr_stream_kernel(const __grid_constant__ Args a, const uint32_t stage_bytes) {
    constexpr int kW = Stream<kBack>::kWarps;
    constexpr int kRows = 32 / LANES;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kW][2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = (lane % LANES) * 8, sub = lane / LANES;
    const bool live = e0 < a.D;
    const uint32_t tokens = uint32_t(a.B) * uint32_t(a.T), step = gridDim.x * kW;
    uint8_t* mine = smem + warp * 2 * stage_bytes;
    if (lane == 0) {
        tc::mbar_init(tc::smem_u32(&full[warp][0]), 1);
        tc::mbar_init(tc::smem_u32(&full[warp][1]), 1);
        tc::mbar_fence_init();
    }
    __syncwarp();
    const uint32_t row_q = a.Hq * a.D * sizeof(T), row_k = a.Hk * a.D * sizeof(T), row_t = a.R * 4;
    // stage s <- tensor `side` of token n, whose position is p
    auto fetch = [&](uint32_t n, int side, int p, int s) {
        if (tc::elect()) {
            int b, t;
            place(a, n, b, t);
            const uint32_t bar = tc::smem_u32(&full[warp][s]), at = tc::smem_u32(mine + s * stage_bytes), row = side ? row_k : row_q;
            tc::mbar_expect_tx(bar, row * (kBack ? 2 : 1) + row_t);
            tc::bulk_load(at, row_in<T>(a, !side, b, t, 0), row, bar);
            if (kBack) tc::bulk_load(at + row, static_cast<const T*>(side ? a.gk : a.gq) + row_at(a, !side, n, 0), row, bar);
            if (row_t) tc::bulk_load(at + (kBack ? 2 : 1) * row, a.table + int64_t(p < 0 ? 0 : p) * a.R, row_t, bar);
        }
        __syncwarp();
    };
    auto position_of = [&](uint32_t n) {
        int b, t;
        place(a, n, b, t);
        return position(a, b, t);
    };
    uint64_t dw[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[0][i] = dw[1][i] = 0;
    const float inv = mean_factor(a);
    uint32_t n = blockIdx.x * kW + warp;
    int p = 0, ahead = 0;  // positions of this token and the next
    if (n < tokens) {
        p = position_of(n);
        fetch(n, 0, p, 0);
        fetch(n, 1, p, 1);
        if (n + step < tokens) ahead = position_of(n + step);
    }
    uint32_t phase = 0;
    for (; n < tokens; n += step, phase ^= 1) {
#pragma unroll
        for (int side = 0; side < 2; ++side) {  // q in stage 0, k in stage 1
            const int heads = side ? a.Hk : a.Hq;
            const float* wt = side ? a.wk : a.wq;
            const uint32_t row = side ? row_k : row_q;
            const uint8_t* at = mine + side * stage_bytes;
            tc::mbar_wait(tc::smem_u32(&full[warp][side]), phase);
            __syncwarp();
            Turn<T, LANES, kInter, true> turn;
            turn.load(a, reinterpret_cast<const float*>(at + (kBack ? 2 : 1) * row), p < 0, e0, lane);
            uint64_t w[4];
            if (kBack) {
                turn.transpose();
                weights(wt, live, e0, w);
            } else if (wt != nullptr && live) {
                load_pairs(wt + e0, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    turn.c[i] = mul2(turn.c[i], w[i]);
                    turn.s[i] = mul2(turn.s[i], pair(__ldg(wt + turn.partner(a, e0 + 2 * i)), __ldg(wt + turn.partner(a, e0 + 2 * i + 1))));
                }
            }
            T* to = static_cast<T*>(side ? a.ko : a.qo) + row_at(a, !side, n, sub) + e0;
            const T* from = reinterpret_cast<const T*>(at) + sub * a.D + e0;
            const int left = live ? heads - sub : 0, stride = kRows * a.D;
            const bool whole = a.D == LANES * 8 && heads % kRows == 0;  // no lane is ever idle
#pragma unroll 4
            for (int h0 = 0; h0 < heads; h0 += kRows, to += stride, from += stride) {
                const bool on = whole || h0 < left;
                Raw<T> x;
                if (!whole) x.zero();
                if (on) x.shared(from);
                uint64_t v[4], o[4];
                x.pairs(v);
                if (!kBack) {
                    turn.partners(a, x, v, e0, nullptr, o);
                    uint64_t r = both(1.f);
                    if (a.norm) {
                        uint64_t sq = mul2(v[0], v[0]);
#pragma unroll
                        for (int i = 1; i < 4; ++i) sq = fma2(v[i], v[i], sq);
                        r = both(norm_scale(a, row_sum<LANES>(sq), inv));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = mul2(r, fma2(o[i], turn.s[i], mul2(v[i], turn.c[i])));
                    if (on) store8(to, v);
                } else {
                    Raw<T> dy;
                    if (!whole) dy.zero();
                    if (on) dy.shared(from + heads * a.D);
                    uint64_t d[4];
                    dy.pairs(d);
                    turn.partners(a, dy, d, e0, nullptr, o);
                    uint64_t dv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d[i] = fma2(o[i], turn.s[i], mul2(d[i], turn.c[i]));
                        dv[i] = mul2(d[i], v[i]);
                        d[i] = mul2(d[i], w[i]);
                    }
                    uint64_t r2 = both(1.f);
                    if (a.norm) {
                        uint64_t sq = mul2(v[0], v[0]), ux = mul2(dv[0], w[0]);
#pragma unroll
                        for (int i = 1; i < 4; ++i) sq = fma2(v[i], v[i], sq), ux = fma2(dv[i], w[i], ux);
                        const float ss = row_sum<LANES>(sq), r = on ? norm_scale(a, ss, inv) : 0.f, m = r * (r * row_sum<LANES>(ux)) * inv;
                        r2 = both(r);
                        const uint64_t m2 = both(-m);
#pragma unroll
                        for (int i = 0; i < 4; ++i) d[i] = mul2(r2, fma2(v[i], m2, d[i]));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) dw[side][i] = fma2(dv[i], r2, dw[side][i]);
                    if (on) store8(to, d);
                }
            }
            __syncwarp();  // the stage has been read
            if (n + step < tokens) fetch(n + step, side, ahead, side);
        }
        p = ahead;
        if (uint64_t(n) + 2 * uint64_t(step) < tokens) ahead = position_of(n + 2 * step);
    }
    if constexpr (kBack) {
        if (a.part == nullptr) return;
        float x[2][8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                uint32_t u, v;
                unpair(dw[which][i], u, v);
                x[which][2 * i] = __uint_as_float(u), x[which][2 * i + 1] = __uint_as_float(v);
            }
        __syncthreads();  // every warp is done with its stages
        float* sum = reinterpret_cast<float*>(smem);  // [warp][2][LANES * 8]
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
#pragma unroll
                for (int o = LANES; o < 32; o <<= 1) x[which][i] += __shfl_xor_sync(kAll, x[which][i], o);
                if (sub == 0) sum[(warp * 2 + which) * LANES * 8 + e0 + i] = x[which][i];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.D; i += kW * 32) {
            const int which = i / a.D, e = i % a.D;
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < kW; ++w) y += sum[(w * 2 + which) * LANES * 8 + e];
            a.part[(int64_t(blockIdx.x) * 2 + which) * a.D + e] = y;
        }
    }
}

__global__ void read_flag_kernel(int* out, int clear) {
    *out = tc::g_timeout_flag;
    if (clear) tc::g_timeout_flag = 0;
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

// Warps of a set of 32 / lanes tokens: one where the sets alone fill the multiprocessors (a token's
// cos and sin are then read once), else up to as many as there are groups of heads.
int64_t sets_of(const Args& a, int lanes) { return (int64_t(a.B) * a.T * lanes + 31) / 32; }
int split_of(const Args& a, int lanes, int unroll) {
    const int groups = (a.Hq + unroll - 1) / unroll + (a.Hk + unroll - 1) / unroll;
    const int64_t want = int64_t(tc::sm_count()) * 32, sets = sets_of(a, lanes);
    if (sets >= want) return 1;
    const int64_t s = (want + sets - 1) / sets;
    return int(s < groups ? s : groups);
}

template <typename T, int LANES, bool kInter, bool kFast, int kU>
void launch_forward(Args a, cudaStream_t s) {
    a.split = split_of(a, LANES, kU);
    const int64_t items = sets_of(a, LANES) * a.split;
    qkr_forward_kernel<T, LANES, kInter, kFast, kU>
        <<<unsigned((items + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a);
}

// The streaming kernel: heads side by side, rows of a token worth a copy that fit a stage, and more
// tokens than the grid has warps.
template <typename T, int LANES, bool kInter, bool kBack>
bool stream(const Args& a, int* blocks, cudaStream_t s) {
    using S = Stream<kBack>;
    const uint32_t bytes = (S::stage(a, sizeof(T)) + 127) / 128 * 128;
    const int rows = 32 / LANES, few = a.Hq < a.Hk ? a.Hq : a.Hk, grid = tc::sm_count() * S::kBlocks;
    const int64_t tokens = int64_t(a.B) * a.T;
    if ((a.Hq > 1 && a.qs[2] != a.D) || (a.Hk > 1 && a.ks[2] != a.D) || bytes > S::kMost || few < 2 * rows ||
        few * a.D * int(sizeof(T)) < 1024 || tokens < 2 * int64_t(grid) * S::kWarps || (kBack && grid > *blocks))
        return false;
    auto f = qkr_stream_kernel<T, LANES, kInter, kBack>;
    size_t smem = size_t(bytes) * 2 * S::kWarps;
    if (kBack && smem < size_t(S::kWarps) * 2 * LANES * 8 * 4) smem = size_t(S::kWarps) * 2 * LANES * 8 * 4;
    if (!tc::set_smem(f, smem)) return false;
    f<<<grid, S::kWarps * 32, smem, s>>>(a, bytes);
    *blocks = grid;
    return true;
}

template <typename T, int LANES, bool kInter, bool kFast>
void launch(Args a, bool back, int* blocks_used, cudaStream_t s) {
    const int blocks = *blocks_used;
    if (kFast && (back ? stream<T, LANES, kInter, true>(a, blocks_used, s) : stream<T, LANES, kInter, false>(a, blocks_used, s))) return;
    // Forward: groups of heads once the tokens give every multiprocessor a warp; below, one head at a time, for
    // more warps a token.  us, groups / single heads, 32 + 8 and 8 + 4 heads of 128 in bf16:
    //     64 tokens      8.8 / 6.8      8.8 / 6.8
    //     1024 tokens    15 / 17        9.8 / 11
    //     2048 tokens    21 / 23        11 / 15
    if (back) {
        a.split = min(split_of(a, LANES, 2), blocks * kWarps);
        qkr_backward_kernel<T, LANES, kInter, kFast><<<blocks, kWarps * 32, 0, s>>>(a);
    } else if (kFast && a.Hq >= 4 && sets_of(a, LANES) >= tc::sm_count()) {
        launch_forward<T, LANES, kInter, kFast, !kFast ? 1 : sizeof(T) == 4 ? 2 : 4>(a, s);
    } else {  // one head at a time, for more warps a token
        launch_forward<T, LANES, kInter, kFast, 1>(a, s);
    }
}

template <typename T, int LANES>
void pick_layout(const Args& a, bool back, int* blocks, cudaStream_t s) {
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
void pick_lanes(const Args& a, bool back, int* blocks, cudaStream_t s) {
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

rm_status run(const rm_cp_qkr_problem* p, const Args& a, bool back, int* blocks, cudaStream_t s) {
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

namespace rmcp {
rm_status qkr_read_timeout_flag(int* host_flag, int clear, int* dev_scratch, cudaStream_t s) {
    qkr::read_flag_kernel<<<1, 1, 0, s>>>(dev_scratch, clear);
    if (!launch_ok()) return RM_ERR_CUDA;
    note_launch(1);
    if (cudaMemcpyAsync(host_flag, dev_scratch, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return RM_ERR_CUDA;
    return cudaStreamSynchronize(s) == cudaSuccess ? RM_OK : RM_ERR_CUDA;
}
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
    int none = 0;
    return rmcp::qkr::run(p, a, false, &none, reinterpret_cast<cudaStream_t>(stream));
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
    int blocks = rmcp::qkr::backward_blocks(int64_t(a.B) * a.T);  // those that left partial sums
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    rmcp::begin_launches();
    st = rmcp::qkr::run(p, a, true, &blocks, s);
    if (st != RM_OK || !weights) return st;
    rmcp::qkr::qkr_weight_kernel<<<dim3(a.D / 8, 2), 256, 0, s>>>(a.part, blocks, a.D, dwq, dwk);
    rmcp::note_launch(1);
    if (!rmcp::launch_ok()) return rmcp::api_fail(RM_ERR_CUDA, "weight gradient launch failed");
    return RM_OK;
}

}  // extern "C"
