// Pages of the 8-bit key/value cache moved in every layer at once: kept drafts
// to the front of their slots (compact), sequences continued by others (fork).
//
// Compact.  One wave per (sequence, kv head, K or V, layer) goes through the
// pages that receive tokens in order.  A kept token's slot is at or behind the
// place that it goes to, and a wave reads a group of tokens before it writes
// them, so nothing is overwritten before it is read.  A page's scale follows the
// append's rule, in whole numbers: code c of a page with exponent byte b asks for
// the byte b + k(c), k the least whole number with |e4m3(c)| <= 448 2^k.
// Bound by latency (one user's 12 drafts in 12 layers 6 us: lengths, path, pages, codes) or by whole lines: a token's
// values lie one in each line of its page, so that 64 users' kept drafts (4 MB of codes) touch 100 MB, 32 us, 20
// at a large copy's rate.  All tokens of a page find their sources at once, a token a lane (46 us one after the other).
//
// Fork.  One workgroup decides everything about the tables: which entries of a
// row are shared, kept or new, the counts, and the lowest free pages for the new
// ones, numbered by row and entry; then any number of workgroups copy pages.
// The tables take 5 to 6 us, a chain of passes over LDS between barriers of one workgroup (33 us with counts in
// device memory and the device's fences); 12 layers' open pages of 64 beams, 63 MB read and written, 11 us behind them.
// That holds for tables of up to a thousand entries.  The workgroup goes through all sequences' entries three times,
// 1024 at once: 32 sequences of 128 entries take 11 us, of 512 25, 128 of 512 (a tenth of them filled) 41.  Past 16384
// pages or 1024 rows the counts are in device memory, some 5 times as slow: 64 sequences of 512 entries on 29576
// pages 130 us, 128 on 59144 256 (kernel trace).
#include "q8_device.hpp"
#include "q8_kv.hpp"

namespace q8 {
namespace {

// The least k with |e4m3(c)| <= 448 2^k, c a code's 7 magnitude bits (1 .. 126)
__device__ __forceinline__ int code_scale(int c) {
  // 448 = 1.75 2^8: a normal code 2^(x - 7) (1 + m / 8) asks for x - 15, one more where m is 7; a subnormal
  // one, m 2^-9 = 2^(h - 9) (1 + f), f at most 0.75, for h - 17
  const int x = c >> 3, m = c & 7;
  return x > 0 ? x - 15 + (m == 7 ? 1 : 0) : 14 - __builtin_clz(m);
}
// The exponent byte that a code of a page with byte b asks for; 0 for zeros and NaN codes
__device__ __forceinline__ int wanted(int c, int b) {
  c &= 0x7f;
  if (c == 0 || c == 0x7f) return 0;
  const int w = b + code_scale(c);
  return w < 0 ? 0 : w;
}
// The largest magnitude among four codes, NaN codes aside (as they order)
__device__ __forceinline__ int largest4(uint32_t w, int most) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = (int)(w >> (8 * i)) & 0x7f;
    most = c != 0x7f && c > most ? c : most;
  }
  return most;
}
// Four codes times 2^shift, NaN codes as they are
__device__ __forceinline__ uint32_t rescaled4(uint32_t w, int shift) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  const uint32_t t = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u, nan = (t << 1) - (t >> 7);
  return (pack4_e4m3(__builtin_ldexpf(lo[0], shift), __builtin_ldexpf(lo[1], shift), __builtin_ldexpf(hi[0], shift),
                     __builtin_ldexpf(hi[1], shift)) & ~nan) | (w & nan);
}
__device__ __forceinline__ int wave_max_i(int v) {
  v = dpp_row_reduce(v, [](int a, int b) { return a > b ? a : b; });
  const int a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const int c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  const int x = a > b ? a : b, y = c > d ? c : d;
  return x > y ? x : y;
}

// The kept path of a sequence as far as it is one: entries i, keep[i] from i on, growing, below n.  Returns
// their number; `stay` receives how many are in place at its front.
__device__ __forceinline__ int path_of(const int32_t* keep, int width, int most, int n, int lane, int* stay) {
  int total = 0, still = 0;
  for (int base = 0;; base += 64) {
    const int i = base + lane;
    // (read before the count is known)
    const int k = i < width ? keep[i] : -1, before = i > 0 && i < width ? keep[i - 1] : -1;
    const bool in = i < most;
    const uint64_t ok = __ballot(in && k >= i && k < n && k > before), same = __ballot(in && k == i);
    const int run = ok == ~0ull ? 64 : __builtin_ctzll(~ok);
    const uint64_t mine = run == 64 ? ~0ull : ((uint64_t)1 << run) - 1, off = mine & ~same;
    if (still == base) still += off ? __builtin_ctzll(off) : run;
    total += run;
    if (run < 64) break;
  }
  *stay = still;
  return total;
}

// Byte e of a word as a value
template <int E>
__device__ __forceinline__ float value_of(uint32_t w) { return __builtin_amdgcn_cvt_f32_fp8((int)w, E); }

// Four codes, each times a power of two of its own, NaN codes as they are
__device__ __forceinline__ uint32_t rescaled4(uint32_t w, const int* shift) {
  const uint32_t t = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u, nan = (t << 1) - (t >> 7);
  return (pack4_e4m3(__builtin_ldexpf(value_of<0>(w), shift[0]), __builtin_ldexpf(value_of<1>(w), shift[1]),
                     __builtin_ldexpf(value_of<2>(w), shift[2]), __builtin_ldexpf(value_of<3>(w), shift[3])) & ~nan) | (w & nan);
}

// Where a page's tokens come from, token i at lane i % 64 of one of two sets (a page has 128 tokens at
// most): page x head, -1 without one; place in that page; its exponent byte.
struct Sources {
  int ph[2], off[2], b[2];
};

template <int D>
__device__ void compact_item(const CompactArgs& a, const CacheLayer& layer, int s, int head, bool is_v, int lane, bool says) {
  const KvView& kv = a.kv;
  const int page_log2 = 31 - __builtin_clz(kv.page), page = kv.page;
  int end = kv.q_start[s + 1], first = kv.q_start[s];
  end = end < 0 ? 0 : end;
  first = first < 0 ? 0 : (first > end ? end : first);
  const int n = end - first, len = kv.kv_len[s] < 0 ? 0 : kv.kv_len[s], past = len - n;
  int most = a.n_keep[s];
  most = most < 0 ? 0 : (most > a.width ? a.width : most);
  const int32_t* const keep = a.keep + (int64_t)s * a.width;
  int stay;
  const int kept = path_of(keep, a.width, most, n, lane, &stay);
  if (says && lane == 0) a.len_out[s] = past + kept < 0 ? 0 : past + kept;
  const int64_t cap = (int64_t)kv.max_pages * page;
  // the slots that receive a token
  int lo = past + stay < 0 ? 0 : past + stay;
  const int hi = past + kept < cap ? past + kept : (int)cap;
  uint8_t* const codes = is_v ? layer.v : layer.k;
  uint8_t* const exps = is_v ? layer.ve : layer.ke;
  const int32_t* const table = kv.table + (int64_t)s * kv.max_pages;
  auto page_at = [&](int slot) {
    if (slot < 0 || slot >= cap) return -1;
    const int p = table[slot >> page_log2];
    return p >= 0 && p < kv.num_pages ? p : -1;
  };
  for (; lo < hi; lo = (lo & ~(page - 1)) + page) {
    const int stop = (lo & ~(page - 1)) + page, top = hi < stop ? hi : stop, count = top - lo;
    // the sources of all tokens in one go, a token a lane
    Sources from{{-1, -1}, {0, 0}, {0, 0}};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 64 * h + lane;
      if (i >= count) continue;
      const int slot = past + keep[lo + i - past], p = page_at(slot);
      if (p < 0) continue;
      from.ph[h] = p * kv.kv_heads + head;
      from.off[h] = slot & (page - 1);
      from.b[h] = exps[from.ph[h]];
    }
    const int to = page_at(lo);
    if (to < 0) continue;
    const int64_t th = (int64_t)to * kv.kv_heads + head;
    uint8_t* const dst = codes + th * page * D;
    const int had = exps[th], old = lo & (page - 1);
    const bool fresh = old == 0;
    int want = -1;
    auto settle = [&] {              // the page's new byte, -1 where nothing comes
      want = wave_max_i(want);
      return want < 0 ? -1 : (fresh || want > had ? want : had);
    };
    if (!is_v) {
      // 16 features a lane, G tokens at once; U of those in registers
      constexpr int C = D / 16, G = 64 / C, U = 2;
      const int c = lane % C;
      v4i x[U];
      int u_b[U];                    // exponent byte; -1: nothing
      auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * G + lane / C;
          int ph = __shfl(from.ph[0], i & 63), off = __shfl(from.off[0], i & 63);
          if (page > 64) {
            const int p1 = __shfl(from.ph[1], i & 63), o1 = __shfl(from.off[1], i & 63);
            ph = i < 64 ? ph : p1;
            off = i < 64 ? off : o1;
          }
          x[u] = v4i{0, 0, 0, 0};
          u_b[u] = -1;
          if (i < count && ph >= 0) {
            x[u] = *(const v4i*)(codes + ((int64_t)ph * page + off) * D + 16 * c);
            u_b[u] = 0;
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * G + lane / C;
          int eb = __shfl(from.b[0], i & 63);
          if (page > 64) {
            const int e1 = __shfl(from.b[1], i & 63);
            eb = i < 64 ? eb : e1;
          }
          u_b[u] = u_b[u] < 0 ? -1 : eb;
        }
      };
      for (int i0 = 0; i0 < count; i0 += U * G) {
        load(i0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u_b[u] < 0) continue;
          int big = 0;
#pragma unroll
          for (int w = 0; w < 4; ++w) big = largest4((uint32_t)x[u][w], big);
          const int w = wanted(big, u_b[u]);
          want = w > want ? w : want;
        }
      }
      const int b = settle();
      if (b < 0) continue;
      if (!fresh && b != had)
        for (int i = lane / C; i < old; i += G) {
          v4i* const p = (v4i*)(dst + i * D + 16 * c);
          v4i y = *p;
#pragma unroll
          for (int w = 0; w < 4; ++w) y[w] = (int)rescaled4((uint32_t)y[w], had - b);
          *p = y;
        }
      for (int i0 = 0; i0 < count; i0 += U * G) {
        if (count > U * G) load(i0);               // (else they are there)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u_b[u] < 0) continue;
          const int shift = u_b[u] - b;
          if (shift != 0)
#pragma unroll
            for (int w = 0; w < 4; ++w) x[u][w] = (int)rescaled4((uint32_t)x[u][w], shift);
          *(v4i*)(dst + (old + i0 + u * G + lane / C) * D + 16 * c) = x[u];
        }
      }
      if (lane == 0 && b != had) exps[th] = (uint8_t)b;
    } else {
      // D / 64 features a lane, U words of four tokens in registers
      constexpr int F = D / 64, U = 2;
      const int w0 = old & ~3, words = (old + count - w0 + 3) / 4;
      uint32_t x[U][F], was[U][F];
      int shift[U][4];               // byte of the token's page; -1: not a new token
      auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int j = 0; j < F; ++j) {
            x[u][j] = 0;
            was[u][j] = i0 + u < words ? *(const uint32_t*)(dst + (lane + 64 * j) * page + w0 + 4 * (i0 + u)) : 0;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = w0 + 4 * (i0 + u) + e - old;       // uniform
            shift[u][e] = -1;
            if (i < 0 || i >= count) continue;
            const int ph = __builtin_amdgcn_readlane(i < 64 ? from.ph[0] : from.ph[1], i & 63);
            const int off = __builtin_amdgcn_readlane(i < 64 ? from.off[0] : from.off[1], i & 63);
            if (ph < 0) continue;
            shift[u][e] = 0;
            const uint8_t* const p = codes + (int64_t)ph * page * D + off;
#pragma unroll
            for (int j = 0; j < F; ++j) x[u][j] |= (uint32_t)p[(lane + 64 * j) * page] << (8 * e);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = w0 + 4 * (i0 + u) + e - old;
            if (shift[u][e] == 0) shift[u][e] = __builtin_amdgcn_readlane(i < 64 ? from.b[0] : from.b[1], i & 63);
          }
      };
      for (int i0 = 0; i0 < words; i0 += U) {
        load(i0);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (shift[u][e] < 0) continue;
#pragma unroll
            for (int j = 0; j < F; ++j) {
              const int w = wanted((int)(x[u][j] >> (8 * e)), shift[u][e]);
              want = w > want ? w : want;
            }
          }
      }
      const int b = settle();
      if (b < 0) continue;
      if (!fresh && b != had)
#pragma unroll
        for (int j = 0; j < F; ++j)
          for (int i = 0; i < w0; i += 4) {
            uint32_t* const p = (uint32_t*)(dst + (lane + 64 * j) * page + i);
            *p = rescaled4(*p, had - b);
          }
      for (int i0 = 0; i0 < words; i0 += U) {
        if (words > U) load(i0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (i0 + u >= words) continue;
          // bytes of new tokens, those before them at the new scale, and what lies between and behind
          uint32_t put = 0;
          int by[4];
          bool move = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool is_new = shift[u][e] >= 0, is_old = w0 + 4 * (i0 + u) + e < old;
            put |= is_new || is_old ? 0xffu << (8 * e) : 0u;
            by[e] = is_new ? shift[u][e] - b : (is_old ? had - b : 0);
            move |= by[e] != 0;
          }
#pragma unroll
          for (int j = 0; j < F; ++j) {
            uint32_t y = x[u][j];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (shift[u][e] < 0) y |= was[u][j] & (0xffu << (8 * e));
            if (move) y = rescaled4(y, by);
            y = (y & put) | (was[u][j] & ~put);
            *(uint32_t*)(dst + (lane + 64 * j) * page + w0 + 4 * (i0 + u)) = y;
          }
        }
      }
      if (lane == 0 && b != had) exps[th] = (uint8_t)b;
    }
  }
}

template <int D>
__global__ __launch_bounds__(256) void k_kv_compact(const CompactArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const CacheLayer& layer = a.layer[blockIdx.y];
  const int64_t items = (int64_t)a.kv.seqs * a.kv.kv_heads * 2;
  for (int64_t i = (int64_t)blockIdx.x * 4 + wave; i < items; i += (int64_t)gridDim.x * 4) {
    const int part = (int)(i % (2 * a.kv.kv_heads)), s = (int)(i / (2 * a.kv.kv_heads));
    compact_item<D>(a, layer, s, part >> 1, part & 1, lane, part == 0 && blockIdx.y == 0 && a.len_out);
  }
}

// ---------------------------------------------------------------------- fork
constexpr int kForkThreads = 1024, kForkWaves = kForkThreads / 64;
constexpr int kNew = -2;           // an entry that waits for its page

// Every thread's v summed over those before it; `all` receives the whole.
__device__ __forceinline__ int block_scan(int v, int* red, int* all) {
  const int wave = threadIdx.x >> 6, incl = wave_incl_scan(v);
  __syncthreads();                 // red is read
  if ((threadIdx.x & 63) == 63) red[wave] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kForkWaves; ++w) {
    before += w < wave ? red[w] : 0;
    total += red[w];
  }
  *all = total;
  return before + incl - v;
}
__device__ __forceinline__ void add_one(int* p, int v) {
  __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

struct Row {
  int parent, len, full, need;     // parent -1: an empty sequence
};
__device__ __forceinline__ Row row_of(const ForkArgs& a, int s) {
  Row r{a.parent[s], 0, 0, 0};
  if (r.parent < 0 || r.parent >= a.seqs) return Row{-1, 0, 0, 0};
  const int64_t cap = (int64_t)a.max_pages * a.page;
  const int len = a.kv_len[r.parent];
  r.len = len < 0 ? 0 : (len < cap ? len : (int)cap);
  r.full = r.len / a.page;
  const int64_t need = (r.len + a.room + a.page - 1) / a.page;
  r.need = need < a.max_pages ? (int)need : a.max_pages;
  return r;
}

// LOCAL: counts and the rows' numbers in LDS (up to kForkPages pages and kForkRows rows of either batch),
// else in the caller's arrays.  A row takes as many lanes as its entries need, up to 64.
constexpr int kForkPages = 16384, kForkRows = 1024;
template <bool LOCAL>
__global__ __launch_bounds__(kForkThreads) void k_kv_fork(const ForkArgs a, int lanes) {
  __shared__ int red[kForkWaves];
  __shared__ int s_count[LOCAL ? kForkPages : 1], s_first[LOCAL ? kForkRows : 1], s_fresh[LOCAL ? kForkRows : 1];
  int* const count = LOCAL ? s_count : a.refs_out;
  int* const first = LOCAL ? s_first : a.first;
  int* const fresh = LOCAL ? s_fresh : a.fresh;
  const int tid = threadIdx.x, lane = tid & 63;
  for (int i = tid; i < a.num_pages; i += kForkThreads) count[i] = a.refs[i];
  for (int i = tid; i < a.seqs; i += kForkThreads) first[i] = a.outs;
  __syncthreads();
  for (int s = tid; s < a.outs; s += kForkThreads) {
    const int p = a.parent[s];
    if (p >= 0 && p < a.seqs) __hip_atomic_fetch_min(&first[p], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  }
  // pages let go
  for (int64_t i = tid; i < (int64_t)a.seqs * a.max_pages; i += kForkThreads) {
    const int e = a.table[i];
    if (e >= 0 && e < a.num_pages) add_one(&count[e], -1);
  }
  __syncthreads();
  // those that rows hold without a new one; a row's lanes start at bit `base` of the wave's
  const int mine = tid / lanes, rows = kForkThreads / lanes, col = tid % lanes, base = lane & ~(lanes - 1);
  const uint64_t whole = lanes == 64 ? ~(uint64_t)0 : (((uint64_t)1 << lanes) - 1) << base;
  const uint64_t below = whole & (((uint64_t)1 << lane) - 1);
  for (int s = mine; s < a.outs; s += rows) {
    const Row r = row_of(a, s);
    const bool heir = r.parent >= 0 && first[r.parent] == s;
    const int32_t* const from = a.table + (int64_t)(r.parent < 0 ? 0 : r.parent) * a.max_pages;
    int news = 0;
    for (int j0 = 0; j0 < a.max_pages; j0 += lanes) {
      const int j = j0 + col;
      int e = -1;
      bool is_new = false;
      if (j < r.need) {
        e = from[j];
        e = e >= 0 && e < a.num_pages ? e : -1;
        if (j >= r.full && !(heir && e >= 0 && a.refs[e] == 1)) {
          is_new = true;
          if (j == r.full && r.len % a.page != 0 && e >= 0) add_one(&count[e], 1);     // held until it is copied
        } else if (e >= 0) {
          add_one(&count[e], 1);
        }
      }
      if (j < a.max_pages) a.table_out[(int64_t)s * a.max_pages + j] = is_new ? kNew : e;
      news += __builtin_popcountll(__ballot(is_new) & whole);
    }
    if (col == 0) fresh[s] = news;
  }
  __syncthreads();
  // new pages are numbered by row and entry
  int all = 0;
  for (int at = 0; at < a.outs; at += kForkThreads) {
    const int s = at + tid, n = s < a.outs ? fresh[s] : 0;
    int sum;
    const int before = block_scan(n, red, &sum);
    if (s < a.outs) fresh[s] = all + before;
    all += sum;
  }
  // and taken from the lowest free ones
  int found = 0;
  for (int64_t at = 0; at < a.num_pages && found < all; at += kForkThreads) {
    const int64_t p = at + tid;
    const bool free = p < a.num_pages && count[p] == 0;
    int sum;
    const int rank = found + block_scan(free ? 1 : 0, red, &sum);
    if (free && rank < all) {
      a.taken[rank] = (int)p;
      count[p] = 1;
    }
    found += sum;
  }
  __syncthreads();
  for (int s = mine; s < a.outs; s += rows) {
    const Row r = row_of(a, s);
    int at = fresh[s], src = -1, dst = -1;
    bool cut = false;
    for (int j0 = 0; j0 < r.need; j0 += lanes) {
      const int j = j0 + col;
      int32_t* const entry = a.table_out + (int64_t)s * a.max_pages + j;
      const bool is_new = j < r.need && *entry == kNew;
      const uint64_t news = __ballot(is_new);
      if (is_new) {
        const int rank = at + __builtin_popcountll(news & below);
        const int page = rank < found && rank < all ? a.taken[rank] : -1;
        *entry = page;
        if (j == r.full && r.len % a.page != 0) {
          const int e = a.table[(int64_t)r.parent * a.max_pages + j];
          cut = page < 0;
          if (e >= 0 && e < a.num_pages) {
            add_one(&count[e], -1);
            src = page >= 0 ? e : -1;
            dst = page;
          }
        }
      }
      at += __builtin_popcountll(news & whole);
    }
    // the lane of the open page has the word, the row's first lane where it has none
    const uint64_t copies = __ballot(src >= 0) & whole, cuts = __ballot(cut) & whole;
    if (copies ? src >= 0 : col == 0) {
      a.len_out[s] = cuts ? r.full * a.page : r.len;
      a.copies[2 * s] = src;
      a.copies[2 * s + 1] = dst;
    }
  }
  if (tid == 0) *a.missing = all > found ? all - found : 0;
  if constexpr (LOCAL) {
    __syncthreads();
    for (int i = tid; i < a.num_pages; i += kForkThreads) a.refs_out[i] = count[i];
  }
}

// Slices of 16 KB of a page's keys and values in every layer
constexpr int kSlice = 16384;
__global__ __launch_bounds__(256) void k_copy_pages(const ForkArgs a, int layers, int slices) {
  const int tid = threadIdx.x;
  const int64_t bytes = a.page_bytes, items = (int64_t)a.outs * layers * slices;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int slice = (int)(i % slices), l = (int)(i / slices % layers), s = (int)(i / slices / layers);
    const int src = a.copies[2 * s], dst = a.copies[2 * s + 1];
    if (src < 0) continue;
    const CacheLayer& c = a.layer[l];
    if (slice == 0)
      for (int h = tid; h < 2 * a.kv_heads; h += 256) {
        uint8_t* const e = h < a.kv_heads ? c.ke : c.ve;
        const int hh = h < a.kv_heads ? h : h - a.kv_heads;
        e[(int64_t)dst * a.kv_heads + hh] = e[(int64_t)src * a.kv_heads + hh];
      }
    const int64_t lo = (int64_t)slice * kSlice, hi = lo + kSlice < 2 * bytes ? lo + kSlice : 2 * bytes;
#pragma unroll 4
    for (int64_t o = lo + 16 * tid; o < hi; o += 16 * 256) {
      uint8_t* const base = o < bytes ? c.k : c.v;
      const int64_t off = o < bytes ? o : o - bytes;
      *(v4i*)(base + (int64_t)dst * bytes + off) = *(const v4i*)(base + (int64_t)src * bytes + off);
    }
  }
}

}  // namespace

hipError_t launch_kv_compact(const CompactArgs& a, int dim, int layers, hipStream_t st) {
  const int64_t items = (int64_t)a.kv.seqs * a.kv.kv_heads * 2, blocks = (items + 3) / 4;
  const dim3 grid((unsigned)(blocks < (1 << 22) ? blocks : 1 << 22), (unsigned)layers);
  switch (dim) {
    case 64: k_kv_compact<64><<<grid, 256, 0, st>>>(a); break;
    case 128: k_kv_compact<128><<<grid, 256, 0, st>>>(a); break;
    default: k_kv_compact<256><<<grid, 256, 0, st>>>(a); break;
  }
  return hipGetLastError();
}

hipError_t launch_kv_fork(const ForkArgs& a, hipStream_t st) {
  int lanes = 1;
  while (lanes < 64 && lanes < a.max_pages) lanes *= 2;
  if (a.num_pages <= kForkPages && a.seqs <= kForkRows && a.outs <= kForkRows)
    k_kv_fork<true><<<1, kForkThreads, 0, st>>>(a, lanes);
  else
    k_kv_fork<false><<<1, kForkThreads, 0, st>>>(a, lanes);
  return hipGetLastError();
}

hipError_t launch_copy_pages(const ForkArgs& a, int layers, hipStream_t st) {
  const int slices = (int)((2 * a.page_bytes + kSlice - 1) / kSlice);
  const int64_t items = (int64_t)a.outs * layers * slices;
  k_copy_pages<<<(unsigned)(items < 16384 ? items : 16384), 256, 0, st>>>(a, layers, slices);
  return hipGetLastError();
}

}  // namespace q8
