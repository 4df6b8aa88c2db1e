// gdr_tri.cuh -- the triangular inverse of a 64-token chunk of the gated delta rule and the row
// scaling of its tiles, shared by the segment walks (gdrtc_kernels.cu) and the carried-state form
// (gdstc_kernels.cu).  Internal linkage in each.
#pragma once

#include "tc_tiles.cuh"

namespace rmcp {
namespace gdrtc {

using namespace tc;

namespace {

constexpr int kD = 64;                 // tokens of a chunk; Dk = Dv of the segment walks
constexpr int kP = kD + 1;             // pitch of the fp32 [64][64] A (and scratch) arrays
constexpr int kQ = kD + 4;             // pitch of the fp32 inverse and its partial sums (16-byte rows)
constexpr size_t kF32Bytes = (kD * kP + 2 * kD * kQ) * sizeof(float);  // A, X, Y

// Row t of a [64][64] bf16 tile times w[t] (times mul), from src into dst:
// 512 chunks of 16 bytes, two a thread (a row's scale does not depend on the
// swizzle).
__device__ __forceinline__ void rows_scaled(const uint8_t* src, uint8_t* dst, const float* w, float mul,
                                            int tid) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int n = tid + 256 * k;
        const int r = n >> 3;
        const uint32_t off = uint32_t(r * 128 + (n & 7) * 16);
        float x[8];
        unpack8(*reinterpret_cast<const uint4*>(src + off), x);
        const float f = mul * w[r];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= f;
        *reinterpret_cast<uint4*>(dst + off) = pack8(x);
    }
}

// Xs = (I + La)^{-1} for the strictly lower La (fp32, pitch kP; Xs and the
// scratch Ys pitch kQ): a unit lower triangular inverse by 16 x 16 blocks.
// The four diagonal blocks by forward substitution with the 16 rows of a
// column in 16 lanes (x_k reaches the rows below it by a shuffle; four columns
// a thread, every thread of the CTA busy), then the blocks below the diagonal
// by their distance from it, X_ij = -X_ii sum_{k=j}^{i-1} A_ik X_kj (Ys holds
// the sums), four adjacent columns a thread so that each loaded A or X entry
// serves four products.  Entries above the diagonal are 0.  All 256 threads of
// the CTA call it.
__device__ __noinline__ void tri_inverse(const float* La, float* Xs, float* Ys) {
    const int tid = threadIdx.x;
    for (int e = tid; e < kD * kD / 4; e += blockDim.x) {  // the six blocks above the diagonal
        const int r = e >> 4, c = (e & 15) * 4;
        if ((c >> 4) > (r >> 4)) *reinterpret_cast<float4*>(Xs + r * kQ + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    {
        // warp w: diagonal block w / 2; lane: row r, column group (w % 2, lane / 16)
        const int w = tid >> 5, lane = tid & 31;
        const int o = 16 * (w >> 1), r = lane & 15, grp = ((w & 1) << 1) | (lane >> 4);
        float x[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = r == 4 * grp + m ? 1.f : 0.f;
        const float* lrow = La + (o + r) * kP + o;
#pragma unroll
        for (int k = 0; k < 15; ++k) {
            const float l = lrow[k];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float xk = __shfl_sync(kFull, x[m], (lane & 16) | k);
                if (r > k) x[m] = fmaf(-l, xk, x[m]);
            }
        }
        *reinterpret_cast<float4*>(Xs + (o + r) * kQ + o + 4 * grp) = make_float4(x[0], x[1], x[2], x[3]);
    }
    __syncthreads();
    for (int dist = 1; dist < 4; ++dist) {
        // thread: block (j + dist, j), row r, columns 4 q .. 4 q + 3 of the block
        const bool act = tid < 64 * (4 - dist);
        const int j = tid >> 6, r = (tid >> 2) & 15, q = tid & 3, i = j + dist;
        if (act) {
            float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
            const float* arow = La + (16 * i + r) * kP;
            const float* xc = Xs + 16 * j + 4 * q;
#pragma unroll 16
            for (int kk = 16 * j; kk < 16 * i; ++kk) {
                const float a = arow[kk];
                const float4 xv = *reinterpret_cast<const float4*>(xc + kk * kQ);
                a0 = fmaf(a, xv.x, a0);
                a1 = fmaf(a, xv.y, a1);
                a2 = fmaf(a, xv.z, a2);
                a3 = fmaf(a, xv.w, a3);
            }
            *reinterpret_cast<float4*>(Ys + (16 * i + r) * kQ + 16 * j + 4 * q) = make_float4(a0, a1, a2, a3);
        }
        __syncthreads();
        if (act) {
            float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
            const float* xrow = Xs + (16 * i + r) * kQ + 16 * i;
            const float* yc = Ys + 16 * i * kQ + 16 * j + 4 * q;
#pragma unroll
            for (int kk = 0; kk < 16; ++kk) {
                const float a = xrow[kk];
                const float4 yv = *reinterpret_cast<const float4*>(yc + kk * kQ);
                a0 = fmaf(a, yv.x, a0);
                a1 = fmaf(a, yv.y, a1);
                a2 = fmaf(a, yv.z, a2);
                a3 = fmaf(a, yv.w, a3);
            }
            *reinterpret_cast<float4*>(Xs + (16 * i + r) * kQ + 16 * j + 4 * q) = make_float4(-a0, -a1, -a2, -a3);
        }
        __syncthreads();
    }
}

// Columns c0..c0+15 of row tau of the inverse (pitch kQ).
__device__ __forceinline__ void xs_row16(const float* Xs, int tau, int c0, float* x) {
    const float* row = Xs + tau * kQ + c0;
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
        const float4 v = *reinterpret_cast<const float4*>(row + e);
        x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
    }
}

}  // namespace
}  // namespace gdrtc
}  // namespace rmcp
