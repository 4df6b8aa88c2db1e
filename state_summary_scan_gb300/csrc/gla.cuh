// gla.cuh -- linear attention with a decay for each head and a carried state, shared by its token
// recurrence (gla_kernels.cu), its chunked form (glatc_kernels.cu) and its host side.  Launch
// arguments and sequences are those of the gated delta rule on a pool (beta is not used).
#pragma once

#include "gds.cuh"

namespace rmcp {
namespace gla {

using gds::Args;
using gds::Seq;
using gds::sequence;
using gds::zero_others;
using gds::zero_outputs;

// The chunked form on the tensor cores, for calls whose longest sequence has this many tokens.  us in a CUDA graph,
// tokens as tiles / chunks (bf16, fp32 state):
//     tokens                               16         24         32         48         64
//     64 sequences, 16 heads, 128 x 128    51 / 61    66 / 62    82 / 62    114 / 64   146 / 64
//     64 sequences, 32 heads, 64 x 256     109 / 179  144 / 181  180 / 178  257 / 187  333 / 177
//     8 sequences, 32 heads, 128 x 128     18 / 20    24 / 20    29 / 20    39 / 21    49 / 21
//     one sequence, 16 heads, 128 x 128    6.0 / 8.1  7.6 / 8.1  9.0 / 8.0  12 / 7.9   15 / 7.8
//     64 sequences, 16 heads, 64 x 64      18 / 44    23 / 45    29 / 46    39 / 48    50 / 43
inline int chunked_len(const Args& a) { return a.Dk == 128 || a.Dv >= 128 ? 32 : 64; }
bool tc_supports(const Args& a, rm_dtype dt);
size_t tc_workspace_bytes(const Args& a);
rm_status tc_launch(const Args& a, rm_dtype state_dt, cudaStream_t s);

}  // namespace gla
}  // namespace rmcp
