#include "gla.cuh"
namespace rmcp {
namespace gla {
bool tc_supports(const Args&, rm_dtype) { return false; }
size_t tc_workspace_bytes(const Args&) { return 16; }
rm_status tc_launch(const Args&, rm_dtype, cudaStream_t) { return RM_OK; }
}  // namespace gla
}  // namespace rmcp
