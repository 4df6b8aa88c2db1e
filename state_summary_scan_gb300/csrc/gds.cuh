// gds.cuh -- launch arguments of the gated delta rule with a carried state, shared by its
// token recurrence (gds_kernels.cu), its chunked form (gdstc_kernels.cu) and its host side.
#pragma once

#include "pairs.cuh"
#include "tc_tiles.cuh"

namespace rmcp {
namespace gds {

struct Args {
    int S, N, max_len;      // sequences, packed tokens, tokens of a sequence that the launch is chosen for
    int H, hdiv, Dk, Dv;    // head h reads the q and k rows of head h / hdiv
    int slots_n;
    int recurrent;          // never in chunks
    int each;               // tokens of every sequence without cu, else 0
    float scale;
    int64_t qs[2], ks[2], vs[2];  // token and head strides (elements)
    int64_t gs, bs;         // token strides of g and beta
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* beta;
    const int32_t* cu;
    const int32_t* slots;
    const uint8_t* fresh;
    void* state;            // [slots_n][H][Dk][Dv]
    void* o;                // [N][H][Dv]
    void* ws;
};

// Zeros in `cols` adjacent outputs (a multiple of 8, at most 8 a thread) of `rows` tokens, os elements apart.
template <typename T>
__device__ __forceinline__ void zero_outputs(T* o, int64_t os, int rows, int cols, int tid, int threads) {
    const int each = cols / 8, step = threads / each;
    if (tid >= step * each) return;
    o += tid % each * 8;
    for (int r = tid / each; r < rows; r += step) {
        uint4* to = reinterpret_cast<uint4*>(o + r * os);
#pragma unroll
        for (int u = 0; u < int(sizeof(T)) / 2; ++u) to[u] = make_uint4(0, 0, 0, 0);
    }
}

// Tokens [begin, begin + len) of a sequence; slot < 0: a padding sequence.
struct Seq {
    int begin, len, slot;
    bool fresh;
};

__device__ __forceinline__ Seq sequence(const Args& a, int i) {
    Seq s;
    int e;
    if (a.cu == nullptr) {
        s.begin = i * a.each;
        e = s.begin + a.each;
    } else {  // ranges are cut to the tokens that there are
        s.begin = min(max(__ldg(a.cu + i), 0), a.N);
        e = min(max(__ldg(a.cu + i + 1), s.begin), a.N);
    }
    s.len = e - s.begin;  // whatever max_len says
    const int slot = a.slots ? __ldg(a.slots + i) : i;
    s.slot = slot >= 0 && slot < a.slots_n ? slot : -1;
    s.fresh = a.fresh != nullptr && __ldg(a.fresh + i) != 0;
    return s;
}

// The outputs of the tokens that no sequence has, those before the first one and after the last one: 0.  o: the
// first of the `cols` columns of token 0.  Called for every sequence.
template <typename T>
__device__ __forceinline__ void zero_others(const Args& a, int i, const Seq& s, T* o, int cols, int tid, int threads) {
    if (a.cu == nullptr) return;
    const int64_t os = int64_t(a.H) * a.Dv;
    if (i == 0 && s.begin > 0) zero_outputs(o, os, s.begin, cols, tid, threads);
    const int end = s.begin + s.len;
    if (i == a.S - 1 && end < a.N) zero_outputs(o + end * os, os, a.N - end, cols, tid, threads);
}

// The chunked form on the tensor cores, for calls whose longest sequence has this many tokens.  Its two
// launches take a chunk of 64 rows however few of them are tokens, and the recurrence grows with the
// tokens (us in a CUDA graph, recurrence / chunks; bf16, fp32 state):
//     tokens                               32          40          48          64
//     64 sequences, 16 heads, 128 x 128    87 / 107    105 / 109   122 / 111   157 / 105
//     64 sequences, 32 heads, 64 x 256     193 / 279   234 / 283   275 / 285   358 / 259
//     8 sequences, 32 heads, 128 x 128     28 / 33     33 / 33     39 / 34     50 / 32
//     one sequence, 16 heads, 128 x 128    10 / 17     12 / 17     14 / 17     17 / 16
constexpr int kChunkedLen = 48;
bool tc_supports(const Args& a, rm_dtype dt);
size_t tc_workspace_bytes(const Args& a);
rm_status tc_launch(const Args& a, rm_dtype state_dt, cudaStream_t s);

}  // namespace gds
}  // namespace rmcp
