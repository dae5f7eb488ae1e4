// Attention of new queries over the paged 8-bit key/value cache.
//
// Few rows (query tokens x the query heads that share a kv head): a workgroup
// takes 16 with one sequence, kv head and share of the keys; its NW waves take
// 64-key tiles in turn and join at the end.  Each wave computes S^T = K Q^T
// with v_mfma_f32_16x16x32 (16 keys x 16 rows), so lane (q, g)
// (q = lane % 16, g = lane / 16) holds scores of row q.  The keys of the four
// 16-key MFMA tiles are dealt so that lane group g ends up with the 16
// consecutive keys 16 g .. 16 g + 15: tile t's row 4 g + i is key 16 g + 4 t + i.
// These are already the B operand of O^T = V^T P^T (contraction over keys), so
// P needs no exchange between lanes, and lane (d, g) of the A operand is 16
// consecutive bytes of a row of the value cache, whose tokens are innermost.
// K and V go from memory to registers to MFMA without LDS, a tile's 8 D + 8 D
// bytes all requested before the first is used: this is bound by the cache's
// bytes (64 sequences of up to 4099 tokens, 32 heads over 8 of 128 features:
// 313 MB in 75 us, 4.2 TB/s; 2 of 120000: 492 MB in 98 + 6 us to join 59 shares
// of each, where a copy reaches 4.9 TB/s); one sequence of 513 keys takes 9.0
// us, a chain of page table, exponents, codes and the waves' join.
//
// e4m3 codes convert to bf16 / f16 exactly (4 significant bits).  The key
// exponent of a page multiplies the scores, the value exponent the softmax
// weights (one factor of each per lane and tile: 32 keys lie in one page), so
// value codes enter the product as they are.  What is rounded to f16 (2^-11 of
// it) is p_j 2^(b_j - e), p_j = 2^(s_j - m): the weight of a key's codes, m and
// e whole numbers that each row holds (m its largest score so far, rounded down;
// sums and differences of them are exact, so moving them leaves no drift).
// While every page that a row sees has |b_j - e| <= gap, e stays and the exponent
// is part of the exponential's argument; elsewhere e is moved so that the largest
// weight so far is about 1 (a wave's slow step, with the softmax sum taken from
// exponentials of its own).  Either way the row's largest weight is at least 2^-1
// and none passes 2^15, so what f16 cannot hold is below 2^-24 of the row's
// largest, and pages that the row's mask hides do not enter at all.  Maximum, sum
// and accumulator are held in 32 bits.
#include <type_traits>
#include <utility>

#include "q8_device.hpp"
#include "q8_kv.hpp"
#include "q8_kv_plan.hpp"

namespace q8 {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

template <int DT>
__device__ __forceinline__ v4f mma16(const v4i a, const v4i b, const v4f c) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Eight e4m3 codes times a power of two as an MFMA operand of DT
template <int DT>
__device__ __forceinline__ v4i widen8(int lo, int hi, float scale) {
  if constexpr (DT == DT_BF16)
    return v4i{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false)),
               __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true)),
               __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false)),
               __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true))};
  else
    return v4i{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, false)),
               __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, true)),
               __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, false)),
               __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, true))};
}

// v 2^e
__device__ __forceinline__ v4f scaled4(const v4f v, int e) {
  return v4f{__builtin_ldexpf(v[0], e), __builtin_ldexpf(v[1], e), __builtin_ldexpf(v[2], e), __builtin_ldexpf(v[3], e)};
}

// 2^(b - 127) as a float for an exponent byte b in [0, 254]
__device__ __forceinline__ float exp_byte(int b) { return __uint_as_float(b > 0 ? (uint32_t)b << 23 : 0x400000u); }

// The whole number e of a row that has seen no key (any page is out of its gap)
constexpr float kNoExp = -65536.0f;

// NaN codes among the values.  A key that some rows of a block see and others do not enters the latter's
// product with weight 0, which a NaN code turns into NaN.  A block whose sums hold a NaN goes through its
// keys once more with such codes cleared, and puts the NaN where rows do see them afterwards; a block
// without one pays for a sum.
//
// A word of codes without its NaN codes under mask (bit 7 of each byte that counts).
__device__ __forceinline__ int without_nan(int x, uint32_t mask) {
  const uint32_t t = (((uint32_t)x & 0x7f7f7f7fu) + 0x01010101u) & mask;
  return x & (int)~((t << 1) - (t >> 7));
}
// NaN into the output of row `row` at position pos (of this split, share [kb0, kb1) of its keys) for the
// features d0 + step i + 0 .. 3 in which a key that it sees, outside [all_lo, all_hi), holds a NaN code.
template <int D>
__device__ __forceinline__ void put_nan(const AttnArgs& a, int s, int head, int64_t row, int pos, int split, bool split_out,
                                        int kb0, int kb1, int all_lo, int all_hi, int d0, int step) {
  const KvView kv = a.kv;
  int low = a.window > 0 ? pos - a.window + 1 : 0, high = a.causal && pos + 1 < kb1 ? pos + 1 : kb1;
  low = low > kb0 ? low : kb0;
  for (int key = low; key < high; ++key) {
    if (key >= all_lo && key < all_hi) {
      key = all_hi - 1;
      continue;
    }
    int p = kv.table[(int64_t)s * kv.max_pages + (key >> (31 - __builtin_clz(kv.page)))];
    p = p < 0 ? 0 : (p >= kv.num_pages ? kv.num_pages - 1 : p);
    const uint8_t* const v = kv.v + ((int64_t)p * kv.kv_heads + head) * D * kv.page + (key & (kv.page - 1));
#pragma unroll 1
    for (int d = d0; d < D; d += (d & 3) == 3 ? step - 3 : 1) {
      if ((v[d * kv.page] & 0x7f) != 0x7f) continue;
      if (split_out) a.part[((int64_t)split * kv.tokens * a.heads + row) * D + d] = __builtin_nanf("");
      else ((uint16_t*)a.out)[row * D + d] = 0x7fff;
    }
  }
}

// The rows of one sequence and the keys any of them sees.
struct Span {
  int first, n;        // tokens [first, first + n) of the batch
  int past, total;     // positions of the first new token; cached tokens
  int klo, khi;        // keys that some row of the block sees, within the table
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int s) {
  const KvView& kv = a.kv;
  Span r;
  int end = kv.q_start[s + 1], first = kv.q_start[s];
  end = end < 0 ? 0 : (end > kv.tokens ? kv.tokens : end);
  first = first < 0 ? 0 : (first > end ? end : first);
  r.first = first;
  r.n = end - first;
  const int len = kv.kv_len[s] < 0 ? 0 : kv.kv_len[s];
  const int64_t cap = (int64_t)kv.max_pages * kv.page;
  r.past = len - r.n;
  r.total = len < cap ? len : (int)cap;
  r.klo = 0;
  r.khi = r.total;
  return r;
}

template <int D, int DT, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void k_attn_rows(const AttnArgs a, int row_tiles, int chunk) {
  constexpr int KS = D / 32;        // MFMA steps over the features
  constexpr int KL = D / 64;        // 16-byte loads of a lane's share of a key
  constexpr int NT = D / 16;        // 16-feature tiles of the output
  // weights p 2^(b - e + kUp), p < 2: the largest from 2^(kUp - kGap) to 2^15
  constexpr float kGap = 7.0f, kUp = 7.0f;
  const KvView& kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int split = blockIdx.x, head = blockIdx.y;
  const int s = blockIdx.z / row_tiles, tile0 = blockIdx.z % row_tiles;
  const int group = a.heads / kv.kv_heads;
  const Span sp = span_of(a, s);
  const int rows = sp.n * group;
  const bool split_out = gridDim.x > 1;
  const int page_log2 = 31 - __builtin_clz(kv.page);

  __shared__ __attribute__((aligned(16))) float s_acc[NW][16][D + 4];
  __shared__ float s_ml[NW][16][2];
  __shared__ int s_nan[NW];

  bool careful = false;              // the row tile is taken again, without NaN codes
  for (int r0 = tile0 * 16; r0 < rows;) {
    // this lane's row and the keys that it sees: [low, high)
    const int row = r0 + lr, rc = row < rows ? row : rows - 1;
    const int tok = rc / group, hq = rc - tok * group;
    const int pos = sp.past + tok;
    int high = a.causal ? (pos + 1 < sp.total ? pos + 1 : sp.total) : sp.total;
    const int low = a.window > 0 ? pos - a.window + 1 : 0;
    if (row >= rows) high = 0;
    // features 64 i + 16 g .. + 15 of the row, as the lane's loads of a key give them
    v4i qf[KS];
    {
      const uint16_t* q = (const uint16_t*)a.q + (int64_t)(sp.first + tok) * a.q_stride +
                          (int64_t)(head * group + hq) * D + 16 * lg;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) qf[ks] = *(const v4i*)(q + 64 * (ks >> 1) + 8 * (ks & 1));
    }
    // keys that any row of the tile sees
    const int last = (r0 + 16 < rows ? r0 + 16 : rows) - 1;
    const int pos0 = sp.past + r0 / group, pos1 = sp.past + last / group;
    const int klo = a.window > 0 && pos0 - a.window + 1 > 0 ? pos0 - a.window + 1 : 0;
    const int khi = a.causal ? (pos1 + 1 < sp.total ? pos1 + 1 : sp.total) : sp.total;
    // those that all of them see, and whether there are others
    const int all_lo = a.window > 0 && pos1 - a.window + 1 > 0 ? pos1 - a.window + 1 : 0;
    const int all_hi = a.causal ? (pos0 + 1 < sp.total ? pos0 + 1 : sp.total) : sp.total;
    const bool mixed = all_lo != klo || all_hi != khi;
    // this workgroup's share: `chunk` keys from a multiple of kTile on, the last share all that is left
    const int base = klo & ~(kTile - 1);
    const int64_t from = (int64_t)split * chunk;
    const int kb0 = base + from < khi ? base + (int)from : khi;
    const int kb1 = split + 1 < (int)gridDim.x && kb0 + (int64_t)chunk < khi ? kb0 + chunk : khi;

    v4f acc[NT];
    float m = -INFINITY, l = 0.0f, e = kNoExp;
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = v4f{0, 0, 0, 0};

    // page of a 32-key half of a tile; one without a visible key reads page 0 and is masked
    auto page_of = [&](int key) {
      const bool ok = key < khi && key + 32 > klo;
      int p = ok ? kv.table[(int64_t)s * kv.max_pages + (key >> page_log2)] : 0;
      return p < 0 ? 0 : (p >= kv.num_pages ? kv.num_pages - 1 : p);
    };
    // A tile in registers.  The next one's is requested before the current one is used, and the pages of
    // the one after that (of the lane's key rows, pk, and of its own 16 keys, pv) beside it.
    struct Tile {
      v4i k[4][KL], v[NT];
      int ke, ve;
    };
    constexpr int kStride = NW * kTile;
    int pk = 0, pv = 0;
    auto pages = [&](int kb) {
      if (kb >= kb1) return;
      pk = page_of(kb + 32 * (lr >> 3));
      pv = page_of(kb + 32 * (lg >> 1));
    };
    auto request = [&](Tile& x, int kb) {
      if (kb >= kb1) return;
      const int keyk = kb + 16 * (lr >> 2), keyv = kb + 16 * lg;
      const int64_t ph_k = (int64_t)pk * kv.kv_heads + head, ph_v = (int64_t)pv * kv.kv_heads + head;
      const uint8_t* const kp = kv.k + (ph_k * kv.page + (keyk & (kv.page - 1)) + (lr & 3)) * D + 16 * lg;
      const uint8_t* const vp = kv.v + (ph_v * D + lr) * kv.page + (keyv & (kv.page - 1));
      pages(kb + kStride);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < KL; ++i) x.k[t][i] = *(const v4i*)(kp + t * 4 * D + 64 * i);
      x.ke = kv.ke[ph_v];
      x.ve = kv.ve[ph_v];
#pragma unroll
      for (int n = 0; n < NT; ++n) x.v[n] = *(const v4i*)(vp + 16 * n * kv.page);
    };
    auto attend = [&](Tile& x, int kb) {
      auto& kx = x.k;
      auto& vx = x.v;
      const int kb8 = x.ke, vb = x.ve;
      const int keyv = kb + 16 * lg;
      v4f sc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        sc[t] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < KL; ++i) {
          sc[t] = mma16<DT>(widen8<DT>(kx[t][i][0], kx[t][i][1], 1.0f), qf[2 * i], sc[t]);
          sc[t] = mma16<DT>(widen8<DT>(kx[t][i][2], kx[t][i][3], 1.0f), qf[2 * i + 1], sc[t]);
        }
      }
      // the scores; register 4 t + i is key keyv + 4 t + i
      const float kscale = exp_byte(kb8) * a.scale_log2;
      const bool edge = kb < klo || kb + kTile > khi, all = kb >= low && kb + kTile <= high;
      float mx = -INFINITY;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = keyv + 4 * t + i;
          const float x = all || (key >= low && key < high) ? sc[t][i] * kscale : -INFINITY;
          sc[t][i] = x;
          mx = fmaxf(mx, x);
        }
      // over the row's four lanes; a lane without a visible key has no say about the exponents
      const bool seen = mx > -INFINITY;
      const float own = ceilf(mx) + (float)vb;
      float gap = seen ? (float)vb - e : 0.0f;
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float mn = fmaxf(m, floorf(mx));
      const float ref = mn == -INFINITY ? 0.0f : mn;
      const float alpha = __builtin_amdgcn_exp2f(m - ref);
      float fix = alpha, share = __builtin_amdgcn_exp2f(-(gap + kUp));
      l *= alpha;
      if (__any(fabsf(gap) > kGap)) {
        // the largest weight of this step is 2^top at most, that of the keys before 2^(m + e) to within the gap
        float top = fmaxf(own, __shfl_xor(own, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float to = mn == -INFINITY ? e : fmaxf(top - mn, e - (mn - m));
        fix = __builtin_amdgcn_exp2f(m - ref + (e - to));
        e = to;
        gap = seen ? (float)vb - e : 0.0f;
        share = 0.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) l += __builtin_amdgcn_exp2f(sc[t][i] - ref);
      }
      m = mn;
      const float wref = ref - (gap + kUp);
      float sum = 0.0f;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc[t][i] = __builtin_amdgcn_exp2f(sc[t][i] - wref);
          sum += sc[t][i];
        }
      l = __builtin_fmaf(sum, share, l);
      v4i pf[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        pf[j] = v4i{(int)pack2_out<DT_F16>(sc[2 * j][0], sc[2 * j][1]), (int)pack2_out<DT_F16>(sc[2 * j][2], sc[2 * j][3]),
                    (int)pack2_out<DT_F16>(sc[2 * j + 1][0], sc[2 * j + 1][1]),
                    (int)pack2_out<DT_F16>(sc[2 * j + 1][2], sc[2 * j + 1][3])};
      if (__any(fix != 1.0f)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n] *= fix;
      }
      if (edge) {
        // codes of keys that no row sees may be anything, NaN included: the values' are cleared
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t keep = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = keyv + 4 * w + i;
            keep |= key >= klo && key < khi ? 0xffu << (8 * i) : 0u;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) vx[n][w] &= (int)keep;
        }
      }
      if (__builtin_expect(careful, 0)) {
        int at = keyv;
        asm volatile("" : "+v"(at));               // nothing of this ahead of the loop
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t some = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = at + 4 * w + i;
            some |= key < all_lo || key >= all_hi ? 0x80u << (8 * i) : 0u;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            vx[n][w] = without_nan(vx[n][w], some);
            __builtin_amdgcn_sched_barrier(0);       // one after the other: the registers are all taken
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[n] = mma16<DT_F16>(widen8<DT_F16>(vx[n][0], vx[n][1], 1.0f), pf[0], acc[n]);
        acc[n] = mma16<DT_F16>(widen8<DT_F16>(vx[n][2], vx[n][3], 1.0f), pf[1], acc[n]);
      }
    };
    Tile one, two;
    int kb = kb0 + wave * kTile;
    pages(kb);
    request(one, kb);
    for (; kb < kb1; kb += 2 * kStride) {
      request(two, kb + kStride);
      __builtin_amdgcn_sched_barrier(0);
      attend(one, kb);
      __builtin_amdgcn_sched_barrier(0);
      if (kb + kStride >= kb1) break;
      request(one, kb + 2 * kStride);
      __builtin_amdgcn_sched_barrier(0);
      attend(two, kb + kStride);
      __builtin_amdgcn_sched_barrier(0);
    }

    // join the waves
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    const int unit = (int)(e - (127.0f + kUp));
    __syncthreads();                 // the row tile before is read
#pragma unroll
    for (int n = 0; n < NT; ++n) *(v4f*)&s_acc[wave][lr][16 * n + 4 * lg] = scaled4(acc[n], unit);
    if (lg == 0) {
      s_ml[wave][lr][0] = m;
      s_ml[wave][lr][1] = l;
    }
    if (mixed) {
      float sum = 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) sum += (acc[n][0] + acc[n][1]) + (acc[n][2] + acc[n][3]);
      const int nan = __any(sum != sum);
      if (lane == 0) s_nan[wave] = nan;
    }
    __syncthreads();
    if (mixed && !careful) {
      int nan = s_nan[0];
#pragma unroll
      for (int w = 1; w < NW; ++w) nan |= s_nan[w];
      careful = nan != 0;
      if (careful) continue;
    }
    // 16 threads per row, each D / 16 features
    int again = tid;               // (what it is split into need not live through the loop)
    asm volatile("" : "+v"(again));
    const int row16 = again >> 4, part = again & 15;
    const int orw = r0 + row16;
    if (again < 256 && orw < rows) {
      float mm = s_ml[0][row16][0];
#pragma unroll
      for (int w = 1; w < NW; ++w) mm = fmaxf(mm, s_ml[w][row16][0]);
      const float ref = mm == -INFINITY ? 0.0f : mm;
      float f[NW], ll = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        f[w] = __builtin_amdgcn_exp2f(s_ml[w][row16][0] - ref);
        ll += f[w] * s_ml[w][row16][1];
      }
      const int otok = orw / group, oh = orw - otok * group;
      const int64_t orow = (int64_t)(sp.first + otok) * a.heads + head * group + oh;
      const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
#pragma unroll
      for (int e = 0; e < D / 64; ++e) {
        const int d = part * 4 + e * 64;
        v4f o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < NW; ++w) o += *(const v4f*)&s_acc[w][row16][d] * f[w];
        if (split_out) {
          *(v4f*)(a.part + ((int64_t)split * kv.tokens * a.heads + orow) * D + d) = o;
        } else {
          o *= inv;
          *(v2i*)((uint16_t*)a.out + orow * D + d) = v2i{(int)pack2_out<DT>(o[0], o[1]), (int)pack2_out<DT>(o[2], o[3])};
        }
      }
      if (__builtin_expect(careful, 0)) put_nan<D>(a, s, head, orow, sp.past + otok, split, split_out, kb0, kb1, all_lo, all_hi, part * 4, 64);
      if (part == 0) {
        if (split_out) {
          float* ml = a.part_ml + ((int64_t)split * kv.tokens * a.heads + orow) * 2;
          ml[0] = mm;
          ml[1] = ll;
        } else if (a.lse) {
          a.lse[orow] = ll == 0.0f ? -INFINITY : (mm + __builtin_amdgcn_logf(ll)) * 0.6931471805599453f;
        }
      }
    }
    careful = false;
    r0 += row_tiles * 16;
  }
}

// ---------------------------------------------------------------- many rows
// A workgroup of NW waves takes 32 NW rows of one sequence and kv head, 32 a
// wave, and goes through the keys in steps of 64.  The codes of a step are read
// once, two steps ahead, widened by the thread that read them and put into
// LDS (two buffers), from where every wave reads MFMA operands; widened by each
// wave for itself the conversions are a third of all vector instructions
// (675 against 657 us for a prompt of 8192 tokens, 32 heads over 8).
//
// v_mfma_f32_32x32x16: S^T = K Q^T in two 32-key tiles, lane (q, h) (q = lane %
// 32, h = lane / 32) holding row q; tile T's row 8 a + 4 h + b is key 32 h +
// 16 T + 4 a + b, so that register i of tile T is key 32 h + 16 T + i and the
// weights are the B operand of O^T = V^T P^T as they stand.
//
// The running maximum is a reference that is only moved when a score passes it
// by 8 (p up to 2^8 costs no precision): most steps neither rescale nor exchange
// anything between lanes.
//
// Bound by the matrix units at the clock that the power leaves them: the prompt
// of 8192 tokens is 550 G flop in 572 us once the clock has settled, 0.96
// PFLOP/s, where a plain 8192^3 product reaches 1.45 (the first 20 launches after
// a pause 655 us, and the product 1.25).  When the whole took 580 us its MFMAs
// alone took 465, with the LDS reads of their operands 494.  Two workgroups of 4
// waves a CU 775 us, halves of the waves in turns 766.
typedef float v16 __attribute__((ext_vector_type(16)));
constexpr int kMeta = 256;       // 32-key halves whose page and exponents are held at a time

template <int DT>
__device__ __forceinline__ v16 mma32(const v4i a, const v4i b, const v16 c) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// f(0) .. f(N - 1) with the number as a type: what it indexes stays in registers
template <typename F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) { each_of(f, std::make_integer_sequence<int, N>{}); }

// b where `mask` is all ones, a where it is 0 (a select the compiler cannot turn into an indexed read)
__device__ __forceinline__ int pick(int mask, int a, int b) { return (a & ~mask) | (b & mask); }

// LDS places of the widened operands: 16-byte chunk c of a key's 2 D bytes (of a feature's 128 bytes
// of values) sits at chunk c ^ key_swz (val_swz), so that the 16 lanes that a ds_read_b128 serves in
// one cycle (0-3, 12-15, 20-23, 24-27 and their complements) cover all 64 banks once.
template <int D>
__device__ __forceinline__ constexpr int key_swz(int key) { return D == 64 ? (key >> 1) & 7 : key & 15; }
__device__ __forceinline__ int val_swz(int d) { return (d >> 1) & 7; }

template <int D, int DT, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void k_attn_tiles(const AttnArgs a, int row_tiles, int splits,
                                                                         int chunk) {
  constexpr int kThr = 64 * NW, kRows = 32 * NW;
  constexpr int KS = D / 16;                     // MFMA steps over the features
  constexpr int NT = D / 32;                     // 32-feature tiles of the output
  constexpr int kTileBytes = kStep * D * 2;      // of widened keys, and of values
  constexpr int kChunks = kStep * D / 16;        // 16-byte chunks of codes of a step's keys, and of its values
  constexpr int kPer = 2 * kChunks / kThr;       // of a thread
  static_assert(kPer >= 1 && 2 * kChunks % kThr == 0 && kChunks % 64 == 0, "load split");
  // weights p 2^(b - e + kUp), p <= 2^8: the largest from 2^(kUp - kGap) to 2^15
  constexpr float kGap = 4.0f, kUp = 3.0f;
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * 2 * kTileBytes];
  // byte offset of the page's head, and the exponent bytes (keys | values << 8), of each 32-key half
  // of up to kMeta / 2 steps
  __shared__ int64_t s_page[kMeta];
  __shared__ int s_exp[kMeta];
  __shared__ int s_nan[NW];
  const KvView& kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 31, lh = lane >> 5;
  // one kv head's workgroups on one XCD where the heads allow it (the dispatcher deals workgroups
  // round-robin over the XCDs), the longest rows first
  int b = blockIdx.x;
  const int head = b % kv.kv_heads;
  b /= kv.kv_heads;
  const int split = b % splits;
  b /= splits;
  const int s = b % kv.seqs, tile0 = b / kv.seqs;
  const int group = a.heads / kv.kv_heads;
  const Span sp = span_of(a, s);
  const int rows = sp.n * group;
  const int tiles = (rows + kRows - 1) / kRows;
  const int page_log2 = 31 - __builtin_clz(kv.page);

  bool careful = false;                          // the tile is taken again, without NaN codes
  for (int tile = tiles - 1 - tile0; tile >= 0;) {
    const int r0 = tile * kRows;
    // this lane's row (rows past the end repeat the last one and are not stored)
    const int row = r0 + 32 * wave + lr, rc = row < rows ? row : rows - 1;
    const int tok = rc / group, hq = rc - tok * group;
    const int pos = sp.past + tok;
    v4i qf[KS];
    {
      int qh = lh;
      asm volatile("" : "+v"(qh));               // (kept out of the loop's registers)
      const uint16_t* q = (const uint16_t*)a.q + (int64_t)(sp.first + tok) * a.q_stride +
                          (int64_t)(head * group + hq) * D + qh * (D / 2);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[ks] = *(const v4i*)(q + 8 * ks);
        if (a.scale_log2 < 0.0f) qf[ks] ^= (int)0x80008000u;      // the sign of the scale goes into q
      }
    }
    const float scale = fabsf(a.scale_log2);
    // keys that any row of the block sees, and those that every row of the wave does
    const int last = (r0 + kRows < rows ? r0 + kRows : rows) - 1;
    const int p0 = sp.past + r0 / group, p1 = sp.past + last / group;
    const int klo = a.window > 0 && p0 - a.window + 1 > 0 ? p0 - a.window + 1 : 0;
    const int khi = a.causal ? (p1 + 1 < sp.total ? p1 + 1 : sp.total) : sp.total;
    const int w0 = r0 + 32 * wave < rows ? r0 + 32 * wave : rows - 1;
    const int w1 = w0 + 31 < rows ? w0 + 31 : rows - 1;
    const int pw0 = sp.past + w0 / group, pw1 = sp.past + w1 / group;
    const int all_hi = a.causal ? (pw0 + 1 < sp.total ? pw0 + 1 : sp.total) : sp.total;
    const int all_lo = a.window > 0 ? pw1 - a.window + 1 : 0;
    // those that every row of the block does, and whether there are others
    const int block_hi = a.causal ? (p0 + 1 < sp.total ? p0 + 1 : sp.total) : sp.total;
    const int block_lo = a.window > 0 && p1 - a.window + 1 > 0 ? p1 - a.window + 1 : 0;
    const bool mixed = block_lo != klo || block_hi != khi;
    const int base = klo & ~(kStep - 1);
    const int64_t from = (int64_t)split * chunk;
    const int kb0 = base + from < khi ? base + (int)from : khi;
    const int kb1 = split + 1 < splits && kb0 + (int64_t)chunk < khi ? kb0 + chunk : khi;
    const int steps = (kb1 - kb0 + kStep - 1) / kStep;

    v16 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = v16{};
    float m = -INFINITY, l = 0.0f, e = kNoExp;

    // chunk j of this thread: codes tid + j threads, the keys' (of step ik) first, then the values' (of iv)
    v4i code[kPer];
    auto is_key = [&](int j) {
      return (j + 1) * kThr <= kChunks ? true : j * kThr >= kChunks ? false : wave * 64 + j * kThr < kChunks;
    };
    // (a step past the run's last is read as the last, and never used)
    auto load_one = [&](auto J, int ik, int iv, int n, int kb_run) {
      constexpr int j = decltype(J)::value;
      const int c = tid + j * kThr;
      if (is_key(j)) {
        ik = ik < n ? ik : n - 1;
        const int key = c / (D / 16), off = (kb_run + ik * kStep + key) & (kv.page - 1);
        code[j] = *(const v4i*)(kv.k + s_page[2 * ik + (key >> 5)] + off * D + c % (D / 16) * 16);
      } else {
        iv = iv < n ? iv : n - 1;
        const int f = (c - kChunks) / 4, kc = (c & 3) * 16, off = (kb_run + iv * kStep + kc) & (kv.page - 1);
        code[j] = *(const v4i*)(kv.v + s_page[2 * iv + (kc >> 5)] + f * kv.page + off);
      }
    };
    auto load = [&](int ik, int iv, int n, int kb_run) {
      each<kPer>([&](auto J) { load_one(J, ik, iv, n, kb_run); });
    };
    // codes of keys that no row sees may be anything, NaN included: the values' are cleared (the scores
    // are masked)
    auto clear = [&](int iv, int kb_run) {
      const int kb = kb_run + iv * kStep;
      if (__builtin_expect(careful, 0)) {
        int first = kb + 16 * (tid & 3);
        asm volatile("" : "+v"(first));          // nothing of this ahead of the loop
        each<kPer>([&](auto J) {
          constexpr int j = decltype(J)::value;
          if (is_key(j)) return;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t some = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = first + 4 * w + e;
              some |= key < block_lo || key >= block_hi ? 0x80u << (8 * e) : 0u;
            }
            code[j][w] = without_nan(code[j][w], some);
          }
        });
      }
      if (kb >= klo && kb + kStep <= khi) return;
      const int first = kb + 16 * (tid & 3);
      each<kPer>([&](auto J) {
        constexpr int j = decltype(J)::value;
        if (is_key(j)) return;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t keep = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = first + 4 * w + e;
            keep |= key >= klo && key < khi ? 0xffu << (8 * e) : 0u;
          }
          code[j][w] &= (int)keep;
        }
      });
    };
    // A lane's two 16-byte writes go out in an order that gives every eight lanes eight different
    // chunk numbers modulo 8 (a ds_write_b128 serves eight lanes a cycle over 32 banks).
    auto put_one = [&](auto J, int ik, int iv) {
      constexpr int j = decltype(J)::value;
      const int x0 = code[j][0], x1 = code[j][1], x2 = code[j][2], x3 = code[j][3];
      const int c = tid + j * kThr;
      if (is_key(j)) {
        const int row = c / (D / 16), src = c % (D / 16);
        const int odd = D > 64 ? (src >> 2) & 1 : 0, swap = -odd;
        uint8_t* const at = smem + (ik & 1) * kTileBytes + row * (2 * D);
        const int place = ((2 * src + odd) ^ key_swz<D>(row)) << 4;
        *(v4i*)(at + place) = widen8<DT>(pick(swap, x0, x2), pick(swap, x1, x3), 1.0f);
        __builtin_amdgcn_sched_barrier(0);
        *(v4i*)(at + (place ^ 16)) = widen8<DT>(pick(swap, x2, x0), pick(swap, x3, x1), 1.0f);
      } else {
        const int row = (c - kChunks) / 4, src = c & 3;
        const int odd = row & 1, swap = -odd;
        uint8_t* const at = smem + (2 + (iv & 1)) * kTileBytes + row * 128;
        const int place = ((2 * src + odd) ^ val_swz(row)) << 4;
        *(v4i*)(at + place) = widen8<DT_F16>(pick(swap, x0, x2), pick(swap, x1, x3), 1.0f);
        __builtin_amdgcn_sched_barrier(0);
        *(v4i*)(at + (place ^ 16)) = widen8<DT_F16>(pick(swap, x2, x0), pick(swap, x3, x1), 1.0f);
      }
    };
    auto put = [&](int ik, int iv) {
      each<kPer>([&](auto J) { put_one(J, ik, iv); });
    };

    // operand row of key tile T: LDS key 32 h' + 16 T + 4 a + b of row 8 a + 4 h' + b
    const int key0 = 32 * ((lr >> 2) & 1) + 4 * (lr >> 3) + (lr & 3);
    const int krow = key0 * (2 * D), kz = key_swz<D>(key0);
    static_assert(key_swz<D>(16) == 0, "both key tiles swizzle alike");
    auto key_op = [&](int i, int x) {              // MFMA x of the scores: key tile x % 2, features x / 2
      return *(const v4i*)(smem + (i & 1) * kTileBytes + krow + (x & 1) * 32 * D + (((lh * KS + (x >> 1)) ^ kz) << 4));
    };
    auto val_op = [&](int i, int x) {              // MFMA x of the output: features x % NT, keys x / NT
      return *(const v4i*)(smem + (2 + (i & 1)) * kTileBytes + (x % NT) * 4096 + lr * 128 +
                           (((4 * lh + x / NT) ^ val_swz(lr)) << 4));
    };
    v16 sc[2], sn[2];
    v4i pf[4];
    float kscale = 0.0f, wref = 0.0f, share = 0.0f;
    auto scores = [&](int i) {
      sn[0] = v16{};
      sn[1] = v16{};
#pragma unroll
      for (int x = 0; x < 2 * KS; ++x) {
        sn[x & 1] = mma32<DT>(key_op(i, x), qf[x >> 1], sn[x & 1]);
        if (x % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto highest = [&] {
      float mx = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, sn[t][r]);
      return mx;
    };
    // the scores of the step at kb (exponents exps, largest mx) become the current ones; `again`: they
    // have been before (the last step's, once more at its end)
    auto settle = [&](int exps, int kb, float mx, bool again) {
      if (!(kb >= all_lo && kb + kStep <= all_hi)) {
        // register 16 t + r is key kb + 32 h + 16 t + r: the row sees those from `low` to below `high`
        const int high = (a.causal ? (pos + 1 < sp.total ? pos + 1 : sp.total) : sp.total) - kb - 32 * lh;
        const int low = (a.window > 0 ? pos - a.window + 1 : 0) - kb - 32 * lh;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r) sn[t][r] = 16 * t + r >= low && 16 * t + r < high ? sn[t][r] : -INFINITY;
        mx = highest();
      }
      // not 0: a masked score of -inf stays one
      kscale = fmaxf(exp_byte(exps & 255) * scale, 1.17549435e-38f);
      mx *= kscale;
      // a lane without a visible key has no say about the exponents
      const bool seen = mx > -INFINITY;
      const float vb = (float)(exps >> 8), own = ceilf(mx) + vb;
      float gap = seen ? vb - e : 0.0f;
      share = __builtin_amdgcn_exp2f(-(gap + kUp));
      if (__any(mx > m + 8.0f || fabsf(gap) > kGap)) {
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float mn = fmaxf(m, floorf(mx)), ref = mn == -INFINITY ? 0.0f : mn;
        float fix = __builtin_amdgcn_exp2f(m - ref);
        l *= fix;
        if (__any(fabsf(gap) > kGap)) {
          // the largest weight of this step is 2^top at most, that of the keys before 2^(m + e) to within
          // the gap
          const float top = fmaxf(own, __shfl_xor(own, 32));
          const float to = mn == -INFINITY ? e : fmaxf(top - mn, e - (mn - m));
          fix = __builtin_amdgcn_exp2f(m - ref + (e - to));
          e = to;
          gap = seen ? vb - e : 0.0f;
          share = 0.0f;
          if (!again) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                l += __builtin_amdgcn_exp2f(__builtin_fmaf(sn[t][r], kscale, -ref));
                asm volatile("" : "+v"(l));        // one after the other: the registers are all taken
              }
          }
        }
        m = mn;
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n] *= fix;
      }
      wref = (m == -INFINITY ? 0.0f : m) - (gap + kUp);
      sc[0] = sn[0];
      sc[1] = sn[1];
    };
    // this wave's LDS accesses are done, then everybody's (the loads of codes stay in flight)
    auto meet = [&] {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(kLgkmcnt0);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };

    for (int run = 0; run < steps; run += kMeta / 2) {
      const int n = steps - run < kMeta / 2 ? steps - run : kMeta / 2;
      const int kb_run = kb0 + run * kStep;
      __syncthreads();                           // the run before is read
      if (tid < kMeta) {
        // a half that no row sees reads page 0
        const int key = kb_run + 32 * tid;
        const bool seen = key < khi && key + 32 > klo;
        int p = seen ? kv.table[(int64_t)s * kv.max_pages + (key >> page_log2)] : 0;
        p = p < 0 ? 0 : (p >= kv.num_pages ? kv.num_pages - 1 : p);
        p = p * kv.kv_heads + head;
        s_page[tid] = (int64_t)p * (kv.page * D);
        s_exp[tid] = kv.ke[p] | kv.ve[p] << 8;
      }
      __syncthreads();
      // Step i multiplies the next step's scores beside its own softmax and puts the codes of the steps
      // after into the buffers that step i - 1 has left.
      load(0, 0, n, kb_run);
      put(0, 0);
      load(1, 0, n, kb_run);
      clear(0, kb_run);
      put(1, 0);
      meet();
      scores(0);
      settle(s_exp[lh], kb_run, highest(), false);
      load(2, 1, n, kb_run);
      meet();
      for (int i = 0; i < n; ++i) {
        const int next = i + 1 < n ? i + 1 : n - 1;
        clear(next, kb_run);
        // Slot x: one MFMA of the next scores, the read of the operand four MFMAs on, and a share of the
        // softmax; then one MFMA of the output, a read, and a share of the search for the next maximum.
        // The order is pinned: left to itself the compiler moves the softmax away from the MFMAs and
        // waits for every read in front of its MFMA.
        constexpr int kAheadOps = 4, kKeyOps = 2 * KS, kValOps = 4 * NT;
        constexpr int kShare = 32 / kKeyOps, kSeek = 32 / kValOps;
        static_assert(kKeyOps % kAheadOps == 0, "the ring of operands runs on from the keys' to the values'");
        const int exps = s_exp[2 * next + lh];
        v4i op[kAheadOps];
#pragma unroll
        for (int x = 0; x < kAheadOps; ++x) op[x] = key_op(i + 1, x);
        sn[0] = v16{};
        sn[1] = v16{};
        float sum = 0.0f, mx = -INFINITY;
        __builtin_amdgcn_sched_barrier(0);
        each<kKeyOps>([&](auto X) {
          constexpr int x = decltype(X)::value;
          sn[x & 1] = mma32<DT>(op[x % kAheadOps], qf[x >> 1], sn[x & 1]);
          op[x % kAheadOps] = x + kAheadOps < kKeyOps ? key_op(i + 1, x + kAheadOps) : val_op(i, x + kAheadOps - kKeyOps);
#pragma unroll
          for (int e = x * kShare; e < (x + 1) * kShare; ++e) {
            const int t = e >> 4, r = e & 15;
            sc[t][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][r], kscale, -wref));
            sum += sc[t][r];
            if ((e & 7) == 7)
              pf[e >> 3] = v4i{(int)pack2_out<DT_F16>(sc[t][r - 7], sc[t][r - 6]), (int)pack2_out<DT_F16>(sc[t][r - 5], sc[t][r - 4]),
                               (int)pack2_out<DT_F16>(sc[t][r - 3], sc[t][r - 2]), (int)pack2_out<DT_F16>(sc[t][r - 1], sc[t][r])};
          }
          asm volatile("" : "+v"(sum));
          __builtin_amdgcn_sched_barrier(0);
        });
        l = __builtin_fmaf(sum, share, l);
        each<kValOps>([&](auto X) {
          constexpr int x = decltype(X)::value;
          acc[x % NT] = mma32<DT_F16>(op[x % kAheadOps], pf[x / NT], acc[x % NT]);
          if constexpr (x + kAheadOps < kValOps) op[x % kAheadOps] = val_op(i, x + kAheadOps);
#pragma unroll
          for (int e = x * kSeek; e < (x + 1) * kSeek; ++e) mx = fmaxf(mx, sn[e >> 4][e & 15]);
          asm volatile("" : "+v"(mx));
          __builtin_amdgcn_sched_barrier(0);
          // the codes that have arrived into LDS, the next ones requested, spread over the slots
          each<kPer>([&](auto J) {
            if constexpr (x == (decltype(J)::value + 1) * kValOps / (kPer + 2)) {
              put_one(J, i + 2, i + 1);
              __builtin_amdgcn_sched_barrier(0);
              load_one(J, i + 3, i + 2, n, kb_run);
              __builtin_amdgcn_sched_barrier(0);
            }
          });
        });
        settle(exps, kb_run + next * kStep, mx, i + 1 == n);
        meet();
      }
    }
    if (mixed && !careful) {
      float sum = 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) sum += acc[n][r];
      const int found = __any(sum != sum);
      __syncthreads();                           // the tile before has read its own
      if (lane == 0) s_nan[wave] = found;
      __syncthreads();
      int nan = s_nan[0];
#pragma unroll
      for (int w = 1; w < NW; ++w) nan |= s_nan[w];
      careful = nan != 0;
      if (careful) continue;
    }

    l += __shfl_xor(l, 32);
    // the lane's row again (its place in the output need not live through the loop)
    int again = __lane_id();
    asm volatile("" : "+v"(again));
    const int oh = again >> 5, orw = r0 + 32 * wave + (again & 31);
    if (orw < rows) {
      const int unit = (int)(e - (127.0f + kUp));
      const int otok = orw / group;
      const int64_t orow = (int64_t)(sp.first + otok) * a.heads + head * group + (orw - otok * group);
      const float inv = splits > 1 ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const int d = 32 * n + 2 * r + 4 * oh;
          const v4f o = scaled4(v4f{acc[n][r], acc[n][r + 1], acc[n][r + 2], acc[n][r + 3]} * inv, unit);
          if (splits > 1) *(v4f*)(a.part + ((int64_t)split * kv.tokens * a.heads + orow) * D + d) = o;
          else *(v2i*)((uint16_t*)a.out + orow * D + d) = v2i{(int)pack2_out<DT>(o[0], o[1]), (int)pack2_out<DT>(o[2], o[3])};
        }
      if (__builtin_expect(careful, 0)) put_nan<D>(a, s, head, orow, sp.past + otok, split, splits > 1, kb0, kb1, block_lo, block_hi, 4 * oh, 8);
      if (oh == 0) {
        if (splits > 1) {
          float* ml = a.part_ml + ((int64_t)split * kv.tokens * a.heads + orow) * 2;
          ml[0] = m;
          ml[1] = l;
        } else if (a.lse) {
          a.lse[orow] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
        }
      }
    }
    careful = false;
    tile -= row_tiles;
  }
}

// Joins the splits of a row: one workgroup per row of a sequence.  Its threads
// take 4 features each of every G-th split (G = 1024 / D groups), then join the
// groups through LDS; always in the same order.  Bound by the partial sums' bytes
// and a launch (a row by less than a workgroup: 15 against 7 us for 64 rows of
// 128 features in 59 splits).
template <int D, int DT>
__global__ __launch_bounds__(256) void k_attn_join(const AttnArgs a, int blocks, int splits) {
  constexpr int G = 1024 / D;
  __shared__ float s_f[kMaxSplits], s_top[4], s_sum[4];
  __shared__ __attribute__((aligned(16))) float s_o[G][D];
  const Span sp = span_of(a, blockIdx.x / blocks);
  const int tid = threadIdx.x, wave = tid >> 6;
  const int64_t rows = (int64_t)a.kv.tokens * a.heads, mine = (int64_t)sp.n * a.heads;
  for (int64_t r = blockIdx.x % blocks; r < mine; r += blocks) {
    const int64_t row = (int64_t)sp.first * a.heads + r;
    // thread i: split i's maximum and sum
    float mi = -INFINITY, li = 0.0f;
    if (tid < splits) {
      const float* ml = a.part_ml + (tid * rows + row) * 2;
      mi = ml[0];
      li = ml[1];
    }
    const int g = tid / (D / 4), d = tid % (D / 4) * 4;
    const float top = wave_max(mi);
    __syncthreads();                       // the row before is read
    if ((tid & 63) == 0) s_top[wave] = top;
    __syncthreads();
    const float mm = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
    const float ref = mm == -INFINITY ? 0.0f : mm;
    const float f = __builtin_amdgcn_exp2f(mi - ref);
    s_f[tid] = f;
    float ls = f * li;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) ls += __shfl_xor(ls, o);
    if ((tid & 63) == 0) s_sum[wave] = ls;
    __syncthreads();
    const float ll = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
    v4f o = {0, 0, 0, 0};
#pragma unroll 4
    for (int i = g; i < splits; i += G) o += *(const v4f*)(a.part + (i * rows + row) * D + d) * s_f[i];
    *(v4f*)&s_o[g][d] = o;
    __syncthreads();
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
    if (tid < D) {
      float v = s_o[0][tid];
#pragma unroll
      for (int i = 1; i < G; ++i) v += s_o[i][tid];
      store_out<DT>(a.out, row * D + tid, v * inv);
    }
    if (a.lse && tid == 0) a.lse[row] = ll == 0.0f ? -INFINITY : (mm + __builtin_amdgcn_logf(ll)) * 0.6931471805599453f;
  }
}

template <int D, int DT>
hipError_t launch_dim(const AttnArgs& a, hipStream_t st) {
  const int64_t rows = (int64_t)a.max_q * (a.heads / a.kv.kv_heads);
  const AttnPlan p = attn_plan(rows, D, a.kv.kv_heads, a.kv.seqs, a.max_q, a.max_kv, a.window);
  const int blocks = (int)p.blocks;
  if (p.per == kSmallRows) {
    const dim3 grid((unsigned)p.splits, (unsigned)a.kv.kv_heads, (unsigned)(p.blocks * a.kv.seqs));
    // 8 waves (half as many tiles one after the other: 513 keys, 8 kv heads, 11.0 against 9.2 us) where
    // every workgroup has a CU to itself
    if (D < 256 && (int64_t)grid.x * grid.y * grid.z <= 256) {
      if constexpr (D < 256) k_attn_rows<D, DT, 8><<<grid, 512, 0, st>>>(a, blocks, p.chunk);
    } else {
      k_attn_rows<D, DT, 4><<<grid, 256, 0, st>>>(a, blocks, p.chunk);
    }
  } else {
    const unsigned grid = (unsigned)(p.blocks * a.kv.seqs * a.kv.kv_heads * p.splits);
    if constexpr (D != 128)
      if (p.per == 128) k_attn_tiles<D, DT, 4><<<grid, 256, 0, st>>>(a, blocks, p.splits, p.chunk);
    if constexpr (D != 256)
      if (p.per == 256) k_attn_tiles<D, DT, 8><<<grid, 512, 0, st>>>(a, blocks, p.splits, p.chunk);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t jb = join_blocks(a.max_q, a.heads, a.kv.seqs);
  k_attn_join<D, DT><<<(unsigned)(jb * a.kv.seqs), 256, 0, st>>>(a, (int)jb, p.splits);
  return hipGetLastError();
}
template <int DT>
hipError_t launch_dt(const AttnArgs& a, int dim, hipStream_t st) {
  switch (dim) {
    case 64: return launch_dim<64, DT>(a, st);
    case 128: return launch_dim<128, DT>(a, st);
    default: return launch_dim<256, DT>(a, st);
  }
}

}  // namespace

int attn_splits(int heads, int kv_heads, int dim, int seqs, int64_t max_q, int64_t max_kv, int window) {
  return attn_plan(max_q * (heads / kv_heads), dim, kv_heads, seqs, max_q, max_kv, window).splits;
}

hipError_t launch_attention(const AttnArgs& a, int dt, int dim, hipStream_t st) {
  return dt == DT_F16 ? launch_dt<DT_F16>(a, dim, st) : launch_dt<DT_BF16>(a, dim, st);
}

}  // namespace q8
