// The append with each head of the new keys and queries normalised before it
// is rotated, and positions of the tokens' own (drafted trees).
#include "q8_kv_append.hpp"

namespace q8 {

hipError_t launch_kv_append_norm(const AppendArgs& a, int dt, int dim, hipStream_t st) { return launch_any<true>(a, dt, dim, st); }

}  // namespace q8
