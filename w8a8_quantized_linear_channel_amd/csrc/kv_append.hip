// Append to the paged 8-bit key/value cache: rotate the new keys by their
// position, find each touched (page, head)'s power-of-two scale, store e4m3
// codes, and rotate the queries of the same tokens.
#include "q8_kv_append.hpp"

namespace q8 {

hipError_t launch_kv_append(const AppendArgs& a, int dt, int dim, hipStream_t st) { return launch_any<false>(a, dt, dim, st); }

}  // namespace q8
