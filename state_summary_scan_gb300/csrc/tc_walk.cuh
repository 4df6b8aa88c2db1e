// tc_walk.cuh -- what the walks over a pool's sequences share (gdstc_kernels.cu, glatc_kernels.cu): tensor-memory
// moves and products with an operand in tensor memory, a warp's bounded waits, tensor maps of packed tokens.
#pragma once

#include "gds.cuh"

namespace rmcp {
namespace gds {

using namespace tc;

// internal linkage, as if written in each including translation unit
namespace {

constexpr uint32_t T8 = kTileBytes;  // one [64][64] bf16 tile

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

// [N tokens][heads][D] bf16 with the given token and head strides; boxes of 64 tokens x 64 columns.
bool map_of(CUtensorMap* m, const void* base, int D, int heads, int N, const int64_t* strides) {
    // a dimension of one element may have any stride; the encoder wants a positive multiple of 16 bytes
    const int64_t hs = heads > 1 && strides[1] > 0 ? strides[1] : D, ts = N > 1 && strides[0] > 0 ? strides[0] : int64_t(heads) * D;
    return make_map_strided(m, base, D, heads, N, hs, ts);
}

}  // namespace
}  // namespace gds
}  // namespace rmcp
