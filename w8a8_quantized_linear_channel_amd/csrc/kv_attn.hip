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
#include "q8_attn.hpp"

namespace q8 {
namespace {

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
      if (__builtin_expect(careful, 0)) put_nan<D, false>(a, s, head, orow, sp.past + otok, split, split_out, kb0, kb1, all_lo, all_hi, part * 4, 64, sp.past);
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
      if (p.per == 128) k_attn_tiles<D, DT, 4, false><<<grid, 256, 0, st>>>(a, blocks, p.splits, p.chunk);
    if constexpr (D != 256)
      if (p.per == 256) k_attn_tiles<D, DT, 8, false><<<grid, 512, 0, st>>>(a, blocks, p.splits, p.chunk);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t jb = join_blocks(a.max_q, a.heads, a.kv.seqs);
  k_attn_join<D, DT, false><<<(unsigned)(jb * a.kv.seqs), 256, 0, st>>>(a, (int)jb, p.splits);
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
