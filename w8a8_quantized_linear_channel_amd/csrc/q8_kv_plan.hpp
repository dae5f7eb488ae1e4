// How the launches over the paged cache are cut (host side, no HIP): every
// kernel goes on over what a grid smaller than its work leaves, so a cut is a
// matter of time only.
#pragma once
#include <stdint.h>

namespace q8 {

// Threads of a launch along x that the cuts stay within (a launch takes fewer than 2^32).
constexpr int64_t kMaxThreads = (int64_t)1 << 31;

// ---------------------------------------------------------------- attention
constexpr int kTile = 64;           // keys of a wave's step (few rows)
constexpr int kStep = 64;           // keys of a step (many rows)
constexpr int kMaxSplits = 256;
constexpr int kSmallRows = 16;      // of a workgroup where there are few rows

// How a call is cut: rows of one workgroup, row blocks of a sequence, splits of the keys and keys of
// one split.
struct AttnPlan {
  int64_t per, blocks;
  int splits, chunk;
};
inline AttnPlan attn_plan(int64_t rows, int dim, int kv_heads, int seqs, int64_t max_q, int64_t max_kv, int window) {
  AttnPlan p;
  const int64_t pairs = (int64_t)seqs * kv_heads;
  int64_t seen = max_kv;
  if (window > 0 && window + max_q < seen) seen = window + max_q;
  // Few rows, 16 a workgroup: up to 64, and up to 128 where the blocks of 16 together read no more than
  // half a million keys (8 kv heads of 128 features, this way against many rows': 24 rows on 300 keys
  // 7.7 against 13.7 us, 64 on 110000 127 against 131, 32 sequences of 64 on 2000 64 against 77, 8 of 128
  // on 300 12 against 21, one of 128 on 16000 42 against 34).  256 features, one wave a SIMD and half the
  // bytes in flight: beyond 16 rows only up to a quarter of a million (2 sequences of 128 on 2000 30
  // against 38, of 64 on 10000 76 against 49).
  // Sequences and heads that alone pass a launch of the other kernel: this one's grid has them in y and z.
  const bool few = rows <= kSmallRows || pairs > kMaxThreads / 512 || (dim < 256 && rows <= 64) ||
                   (rows <= 128 && pairs * ((rows + kSmallRows - 1) / kSmallRows) * seen <=
                                       (int64_t)1 << (dim < 256 ? 19 : 18));
  // Many rows: 8 waves (two on a SIMD) share a step's codes; 4 at 256 features, whose accumulators,
  // queries and scores fit a wave only where it has the SIMD's registers to itself, and at 64 features
  // where blocks of 256 rows would leave CUs without one.
  p.per = few ? kSmallRows
          : dim == 256 || (dim == 64 && pairs * ((rows + 255) / 256) < 256) ? 128 : 256;
  p.blocks = (rows + p.per - 1) / p.per;
  const int64_t groups = pairs * p.blocks;
  // keys that a workgroup's rows see
  const int64_t block_q = p.blocks > 1 ? p.per * max_q / rows + 2 : max_q;
  int64_t keys = max_kv;
  if (window > 0 && window + block_q + 2 * kTile < keys) keys = window + block_q + 2 * kTile;
  int64_t want, least;      // splits, and keys of one
  if (p.per == kSmallRows) {
    // Splits to fill the chip, none where the sequences and heads do it alone (64 sequences, 8 kv heads,
    // up to 4099 keys: 74 us whole, 77 + 5 in 1024-key shares), but none longer than 8192 keys either,
    // so that one long sequence among many does not hold up the rest.  A share under 1024 keys costs
    // the join more than it saves.
    want = groups >= 512 ? 1 : 1024 / groups;
    if (want < keys / 8192) want = keys / 8192;
    least = 1024;
  } else {
    // As many as give every CU a workgroup, where the steps that they take off the longest one are worth
    // the join: its launch and the partial sums that it writes and reads back (32-bit, at some 4.5 TB/s).
    // One sequence, 32 heads, 8 kv heads, 128 features, 512 new tokens on 8192: 4 splits 102 us, 8 splits
    // 113; 5 sequences, 8 heads of each, 28 on 920: 6 splits 18 us, none 34; 5 sequences, 4 heads of
    // each, 576 on 61, window 256: 4 splits 36 us, none 31.
    const double step_us = (double)(kStep * p.per * dim) / (64 * 256 * 128) * 1.8;
    const double whole = (double)keys / kStep * step_us, unit = (double)pairs * (double)rows * dim * 8 / 4.5e6;
    want = 256 / groups;
    const int64_t worth = (int64_t)__builtin_sqrt(whole / unit);
    want = want > worth ? worth : want;
    if (want > 1 && whole / want + 5.0 + unit * want > whole) want = 1;
    least = 128;
  }
  want = want > kMaxSplits ? kMaxSplits : want;
  want = want < 1 ? 1 : want;
  int64_t c = ((keys + want - 1) / want + least / 2 - 1) / (least / 2) * (least / 2);
  c = c < least ? least : c;
  p.splits = (int)((keys + c - 1) / c);
  if (p.splits < 1) p.splits = 1;
  p.chunk = (int)(c < (int64_t)1 << 30 ? c : (int64_t)1 << 30);      // (one split has no use for it)
  if (few && p.blocks > 65535 / seqs) p.blocks = 65535 / seqs;
  const int64_t most_blocks = kMaxThreads / (2 * p.per) / (pairs * p.splits);
  if (!few && p.blocks > most_blocks) p.blocks = most_blocks;
  if (p.blocks < 1) p.blocks = 1;
  return p;
}

// Workgroups (256 threads) of a sequence that join its rows' splits.
inline int64_t join_blocks(int64_t max_q, int heads, int seqs) {
  const int64_t rows = max_q * heads, most = kMaxThreads / 256 / seqs;
  return rows < most ? rows : most;
}

// ------------------------------------------------------------------- append
// Workgroups of the pages of `seqs` sequences: seqs x token_blocks where one new token each is expected,
// else seqs x reach (pages of a sequence at a time) x groups (sets of its heads); of the queries: seqs x
// q_blocks.  A call of more sequences than `seqs` is several launches.
struct AppendPlan {
  int64_t token_blocks, reach, groups, q_blocks;
  int seqs, span;    // span: heads of a thread of the queries' workgroups
  int64_t kv_blocks(int n) const { return token_blocks > 0 ? n * token_blocks : n * reach * groups; }
};
// items: (head, K or V) pairs of a workgroup; units: 8-feature units of a query head (0: no queries)
inline AppendPlan append_plan(int seqs, int64_t max_q, int64_t max_pages, int page, int kv_heads, int dim, int heads,
                              int units, int items, int threads) {
  AppendPlan p;
  const int64_t most = kMaxThreads / threads;
  p.groups = (2 * kv_heads + items - 1) / items;
  // one new token each: lanes by head and features instead of patches, of which it would fill one lane
  // in page / 8
  p.token_blocks = max_q == 1 ? ((int64_t)2 * kv_heads * (dim / 8) + threads - 1) / threads : 0;
  const int64_t each = p.token_blocks > 0 ? p.token_blocks : p.groups;
  p.seqs = seqs <= most / each ? seqs : (int)(most / each);
  p.reach = (max_q + page - 2) / page + 1;           // pages that max_q tokens can lie in
  if (p.reach > max_pages) p.reach = max_pages;
  if (p.token_blocks == 0 && p.reach > most / (p.seqs * p.groups)) p.reach = most / (p.seqs * p.groups);
  // heads of a thread: one where there are few tokens (latency), eight that share their angles elsewhere
  p.span = max_q * seqs >= 1024 ? 8 : 1;
  p.q_blocks = 0;
  if (units > 0) {
    const int64_t spans = (heads + p.span - 1) / p.span;
    p.q_blocks = (max_q * units * spans + threads - 1) / threads;
    const int64_t rest = (2 * most - 1 - p.kv_blocks(p.seqs)) / p.seqs;
    if (p.q_blocks > rest) p.q_blocks = rest;
  }
  return p;
}

}  // namespace q8
