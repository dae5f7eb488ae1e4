// Prints how a launch of the attention of drafted trees is cut, for each line "seqs group kv_heads dim max_q
// max_kv window" of the input: rows of a workgroup, splits and keys of a split.
#include <cstdio>

#include "q8_kv_plan.hpp"

int main() {
  long long seqs, group, kv_heads, dim, max_q, max_kv, window;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld", &seqs, &group, &kv_heads, &dim, &max_q, &max_kv, &window) == 7) {
    const q8::AttnPlan p = q8::tree_plan(max_q * group, (int)dim, (int)kv_heads, (int)seqs, max_q, max_kv, (int)window);
    std::printf("%lld %d %d\n", (long long)p.per, p.splits, p.chunk);
  }
  return 0;
}
