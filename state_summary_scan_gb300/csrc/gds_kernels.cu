// gds_kernels.cu -- the gated delta rule with a carried state as a token recurrence in fp32
// (rm_gdr_state_forward): decoding a few tokens for each of many sequences, and every shape
// that the chunked form on the tensor cores does not take.
//
// Per token, S in R^{Dk x Dv}:
//     d = beta (v - e^g S^T k),   o = scale (e^g S^T q + (q.k) d),   S <- e^g S + k d^T
// The columns of S are independent: a CTA owns 32 columns of one sequence's head and keeps them in
// registers over its tokens (Dk / 16 rows x 4 columns a thread, 128 threads); the state is read
// from the pool once and written once, in 128-byte (fp32) pieces of a row.  Several tokens are taken
// four at a time, so that four share one pass over the state, one reduction across the threads and
// one update.
//
// Bound by HBM when decoding one token: the state's read and write are nearly all of the traffic.
// One CTA per 32 columns keeps the loads in flight per thread to 32 registers and gives even one
// sequence of 16 heads 32 or more CTAs.
#include <cstdio>

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
    if (sq.len <= 0 && !(sq.fresh && sq.slot >= 0)) return;  // a fresh empty sequence leaves a zero state
    T* o = static_cast<T*>(a.o) + (int64_t(sq.begin) * a.H + h) * a.Dv + c0;
    const int64_t os = int64_t(a.H) * a.Dv;
    if (sq.slot < 0) {  // padding
        for (int t = warp; t < sq.len; t += 4)
            if (c0 + lane < a.Dv) o[t * os + lane] = from_f32<T>(0.f);
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
    const int cols = a.Dv - c0;
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

template <typename T, typename TS>
bool token_launch(const Args& a, cudaStream_t s) {
    const dim3 grid(unsigned((a.Dv + kCols - 1) / kCols * a.H), unsigned(a.S));
    // a state's traffic bounds single tokens; several are taken four at a time
    const bool one = a.max_len <= 1;
    auto f = a.Dk == 16   ? (one ? gds_token_kernel<T, TS, 16, 1> : gds_token_kernel<T, TS, 16, 4>)
             : a.Dk == 32 ? (one ? gds_token_kernel<T, TS, 32, 1> : gds_token_kernel<T, TS, 32, 4>)
             : a.Dk == 64 ? (one ? gds_token_kernel<T, TS, 64, 1> : gds_token_kernel<T, TS, 64, 4>)
                          : (one ? gds_token_kernel<T, TS, 128, 1> : gds_token_kernel<T, TS, 128, 4>);
    f<<<grid, kTpb, 0, s>>>(a);
    note_launch(1);
    return launch_ok();
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
    a->S = p->num_seqs, a->N = p->num_tokens, a->max_len = p->max_len, a->H = p->H, a->hdiv = p->H / p->qk_heads;
    a->Dk = p->Dk, a->Dv = p->Dv, a->slots_n = p->num_slots, a->scale = p->scale, a->each = 0;
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
    const bool ok = p->dtype == RM_F32 ? (sf ? gds::token_launch<float, float>(a, s) : gds::token_launch<float, __nv_bfloat16>(a, s))
                                       : (sf ? gds::token_launch<__nv_bfloat16, float>(a, s)
                                             : gds::token_launch<__nv_bfloat16, __nv_bfloat16>(a, s));
    if (ok) return RM_OK;
    char msg[256];
    std::snprintf(msg, sizeof(msg), "gated delta rule with a carried state: launch failed: %s", cuda_error_text());
    return api_fail(RM_ERR_CUDA, msg);
}

}  // extern "C"
