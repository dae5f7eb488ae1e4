// Checks how the launches of the attention of drafted trees are cut, over the sizes that the call admits:
// every grid within a launch's limits (gridDim.x * blockDim.x below 2^32, y and z below 65536), nothing below
// one, splits that cover the keys.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "q8_kv_plan.hpp"

namespace {

uint64_t g_state = 88172645463325252ull;
uint64_t next() {
  g_state ^= g_state << 13;
  g_state ^= g_state >> 7;
  return g_state ^= g_state << 17;
}
// 1 .. most, spread over the logarithm, the ends among them
int64_t some(int64_t most) {
  int bits = 0;
  while (bits < 62 && ((int64_t)1 << bits) <= most) ++bits;
  const uint64_t r = next();
  if (r % 16 == 0) return most;
  const int64_t v = (int64_t)(next() >> (64 - (1 + (int)((r >> 8) % bits))));
  return v < 1 ? 1 : (v > most ? most : v);
}

void check(int seqs, int group, int kv_heads, int dim, int64_t max_q, int64_t max_kv, int window) {
  const int heads = group * kv_heads;
  const uint64_t limit = (uint64_t)1 << 32;
  auto no = [&](const char* what) {
    std::printf("%s: %d sequences, %d heads over %d of %d, max_q %lld, max_kv %lld, window %d\n", what, seqs, heads, kv_heads, dim,
                (long long)max_q, (long long)max_kv, window);
    std::exit(1);
  };
  const q8::AttnPlan p = q8::tree_plan(max_q * group, dim, kv_heads, seqs, max_q, max_kv, window);
  if (p.blocks < 1 || p.splits < 1 || p.splits > q8::kMaxSplits || p.chunk < 64 || p.chunk % 64) no("cut");
  if (p.per <= 32) {
    if ((p.per != 16 && p.per != 32) || (p.per == 32 && dim != 128)) no("rows of a workgroup");
    if ((uint64_t)p.splits * 256 >= limit || kv_heads > 65535 || p.blocks * seqs > 65535) no("grid, few rows");
  } else {
    if (p.per != (dim == 256 ? 128 : 256)) no("rows of a workgroup");
    if ((uint64_t)p.blocks * seqs * kv_heads * p.splits * (2 * p.per) >= limit) no("grid, many rows");
  }
  const int64_t jb = q8::join_blocks(max_q, heads, seqs);
  if (jb < 1 || (uint64_t)jb * seqs * 256 >= limit) no("join grid");
  // the append of 16 features a thread: threads, and workgroups of a sequence's pages
  for (int page : {32, 64, 128}) {
    const int tokens = page * dim > 128 * 128 ? 4 : 2, keys = page / tokens * (dim / 16), vals = page / 8 * (dim / 8);
    const int threads = keys > 256 ? keys : 256, ki = threads / (keys > 64 ? keys : 64), vi = threads / (vals > 64 ? vals : 64);
    const int groups = (kv_heads + ki - 1) / ki + (kv_heads + vi - 1) / vi;
    const q8::AppendPlan a = q8::append_plan(seqs, max_q, some(1 << 20), page, kv_heads, dim, heads, dim / 16, 0, threads, groups, 16);
    const int64_t kv = a.kv_blocks(a.seqs);
    if (a.seqs < 1 || a.seqs > seqs || a.reach < 1 || kv < a.seqs || a.q_blocks < 1) no("append cut");
    if ((uint64_t)(kv + a.q_blocks * a.seqs) * threads >= limit || kv + a.q_blocks * a.seqs > INT32_MAX) no("append grid");
    if (max_q == 1 && a.reach != 1) no("append reach");
  }
}

}  // namespace

int main() {
  check(4096, 4, 8, 128, 16384, 16384, 0);
  check(32768, 1, 1024, 256, 1, 1, 0);
  check(32768, 64, 1024, 256, (int64_t)1 << 30, ((int64_t)1 << 31) - 1, 0);
  const int dims[] = {64, 128, 256};
  for (int i = 0; i < 400000; ++i) {
    const int kv_heads = (int)some(1024), group = (int)some(65536 / kv_heads);
    check((int)some(32768), group, kv_heads, dims[next() % 3], some((int64_t)1 << 30), some(((int64_t)1 << 31) - 1),
          next() % 2 ? (int)some((int64_t)1 << 30) : 0);
  }
  std::printf("ok\n");
  return 0;
}
