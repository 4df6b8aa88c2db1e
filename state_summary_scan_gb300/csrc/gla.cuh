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

// The chunked form on the tensor cores, for calls whose longest sequence has this many tokens.
constexpr int kChunkedLen = 48;
bool tc_supports(const Args& a, rm_dtype dt);
size_t tc_workspace_bytes(const Args& a);
rm_status tc_launch(const Args& a, rm_dtype state_dt, cudaStream_t s);

}  // namespace gla
}  // namespace rmcp
