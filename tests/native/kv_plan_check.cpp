// Checks how the launches over the paged cache are cut, over the sizes that the calls admit: every grid
// within a launch's limits (gridDim.x * blockDim.x below 2^32, y and z below 65536), nothing below one,
// splits that cover the keys.
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
[[noreturn]] void fail(const char* what, int seqs, int heads, int kv_heads, int dim, int64_t max_q, int64_t max_kv, int64_t window) {
  std::printf("%s: %d sequences, %d heads over %d of %d, max_q %lld, max_kv %lld, window %lld\n", what, seqs, heads, kv_heads,
              dim, (long long)max_q, (long long)max_kv, (long long)window);
  std::exit(1);
}

void check(int seqs, int group, int kv_heads, int dim, int page, int64_t max_q, int64_t max_kv, int window) {
  const int heads = group * kv_heads;
  const uint64_t limit = (uint64_t)1 << 32;
  auto no = [&](const char* what) { fail(what, seqs, heads, kv_heads, dim, max_q, max_kv, window); };
  const q8::AttnPlan p = q8::attn_plan(max_q * group, dim, kv_heads, seqs, max_q, max_kv, window);
  if (p.blocks < 1 || p.splits < 1 || p.splits > q8::kMaxSplits || p.chunk < 64 || p.chunk % 64) no("cut");
  if (p.per == q8::kSmallRows) {
    if ((uint64_t)p.splits * 512 >= limit || kv_heads > 65535 || p.blocks * seqs > 65535) no("attention grid, few rows");
  } else if ((uint64_t)p.blocks * seqs * kv_heads * p.splits * (2 * p.per) >= limit) {
    no("attention grid, many rows");
  }
  const int64_t jb = q8::join_blocks(max_q, heads, seqs);
  if (jb < 1 || (uint64_t)jb * seqs * 256 >= limit) no("join grid");
  const int patches = page / 8 * (dim / 8), threads = patches > 256 ? patches : 256, items = threads / (patches > 64 ? patches : 64);
  for (int units : {0, dim / 8, dim / 16}) {
    const q8::AppendPlan a = q8::append_plan(seqs, max_q, some(1 << 20), page, kv_heads, dim, heads, units, items, threads);
    const int64_t kv = a.kv_blocks(a.seqs);
    if (a.seqs < 1 || a.seqs > seqs || a.reach < 1 || kv < a.seqs || (units > 0) != (a.q_blocks > 0)) no("append cut");
    if ((uint64_t)(kv + a.q_blocks * a.seqs) * threads >= limit) no("append grid");
    if (max_q == 1 && a.reach != 1) no("append reach");
  }
}

}  // namespace

int main() {
  // one prompt among thousands of sequences
  check(4096, 4, 8, 128, 64, 16384, 16384, 0);
  check(4096, 4, 8, 64, 64, 16384, 16384, 0);
  check(32768, 1, 1024, 256, 128, 1, 1, 0);
  check(32768, 64, 1024, 256, 32, (int64_t)1 << 30, ((int64_t)1 << 31) - 1, 0);
  for (int i = 0; i < 400000; ++i) {
    const int kv_heads = (int)some(1024), group = (int)some(65536 / kv_heads), dims[] = {64, 128, 256}, pages[] = {32, 64, 128};
    check((int)some(32768), group, kv_heads, dims[next() % 3], pages[next() % 3], some((int64_t)1 << 30),
          some(((int64_t)1 << 31) - 1), next() % 2 ? (int)some((int64_t)1 << 30) : 0);
  }
  std::printf("ok\n");
  return 0;
}
