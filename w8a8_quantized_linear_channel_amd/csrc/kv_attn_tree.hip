// Attention of drafted trees over the paged 8-bit key/value cache: a sequence's new
// tokens see the cached keys and those of each other that a mask names.
//
// What differs from a sequence's own attention (kv_attn.hip) are the shapes: some 8
// to 64 tokens times the heads that share a kv head are 32 to 256 rows on a long
// cache, too many for 16 rows a workgroup (every block of 16 reads the codes anew and
// converts them for itself, two thirds of its instructions) and too few for 256.
//
// A wave takes R x 16 rows and 64-key tiles in turn, straight from memory to MFMA as
// k_attn_rows does (there: the operands' layout): a tile's codes are converted once
// for all R.  The keys' registers are requested again as soon as the scores are
// computed, the values' behind the product, so that a tile needs its registers once
// and two waves fit a SIMD: one's conversions and exponentials run beside the other's
// MFMAs.  The running maximum is a reference that is only moved when a score passes
// it by 8, as in k_attn_tiles.
//
// 32 users' drafts on 700 to 4100 keys (88 rows, 8 kv heads, 137 MB of codes): 65 us, in which VALU
// instructions take a good third of each SIMD's cycles and MFMAs a seventh.  Codes that each wave's own DMA puts into
// LDS took as long as these loads, for all that a load of 16 rows looks up 64 lines (72 us both, then); one workgroup of 8
// waves a CU instead of two of 4 took 82: what is left is where a workgroup starts and ends, lengths, pages, codes and
// masks one after another, the turns of a SIMD's two waves, and the longest sequence: its waves take 16 tiles where the
// average has 8.6, and nothing splits it alone.  256 features have one wave a SIMD: 97 us for 16 heads over 4 (the same
// bytes).
#include "q8_attn.hpp"

namespace q8 {
namespace {

// R x 16 rows of a wave: row r0 + 16 r + lr of the sequence's block, 16 lr-lanes by 4 lg-lanes (k_attn_rows).
// weights p 2^(b - e + kUp), p <= 2^8: the largest from 2^(kUp - kGap) to 2^15
constexpr float kTreeGap = 4.0f, kTreeUp = 3.0f;
template <int D, int DT, int R>
struct TreeRows {
  static constexpr int KS = D / 32, NT = D / 16;
  static constexpr bool LW = kOfRounded<DT, true>;
  v4i qf[R][KS];
  v4f acc[R][NT];
  float m[R], l[R], l16[R], e[R];
  int r0, rows, group;               // (rows past the end repeat the last one and are not stored)

  __device__ __forceinline__ int token(int r, int lr) const {
    const int row = r0 + 16 * r + lr;
    return (row < rows ? row : rows - 1) / group;
  }
  __device__ __forceinline__ void start(const AttnArgs& a, const Span& sp, int head, int lr, int lg) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = r0 + 16 * r + lr, rc = row < rows ? row : rows - 1, tok = rc / group;
      const uint16_t* q = (const uint16_t*)a.q + (int64_t)(sp.first + tok) * a.q_stride +
                          (int64_t)(head * group + (rc - tok * group)) * D + 16 * lg;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[r][k] = *(const v4i*)(q + 64 * (k >> 1) + 8 * (k & 1));
        if (a.scale_log2 < 0.0f) qf[r][k] ^= (int)0x80008000u;      // the sign of the scale goes into q
      }
      m[r] = -INFINITY;
      l[r] = l16[r] = 0.0f;
      e[r] = kNoExp;
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[r][n] = v4f{0, 0, 0, 0};
    }
  }
  // The first cached key that each row sees, and its bits of the 16 keys from kb + 16 lg on
  __device__ __forceinline__ void seen(const AttnArgs& a, const Span& sp, int kb, int lr, int lg, int (&low)[R], uint32_t (&bits)[R]) const {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int tok = token(r, lr), at = a.window > 0 ? drafted_at(a, sp.first, tok, sp.past, sp.n) - a.window + 1 : 0;
      low[r] = at < sp.past ? at : sp.past;          // (the window is the cached keys' alone)
      bits[r] = drafted<16>(a.mask + (int64_t)(sp.first + tok) * a.words, a.words, kb + 16 * lg - sp.past);
    }
  }
  // Scores sc of the tile at kb (register 4 t + i is key kb + 16 lg + 4 t + i, exponent bytes exps) to the
  // product's weights pf, the sums and the references with them
  __device__ __forceinline__ void weigh(const AttnArgs& a, const Span& sp, const Keys& ks, int kb, int lr, int lg, int exps, float scale,
                                        const int (&low)[R], const uint32_t (&bits)[R], v4f (&sc)[R][4], v4i (&pf)[R][2]) {
    const int keyv = kb + 16 * lg;
    // not 0: a masked score of -inf stays one
    const float kscale = fmaxf(exp_byte(exps & 255) * scale, 1.17549435e-38f), own_b = (float)(exps >> 8);
    if (!(kb >= ks.all_lo && kb + kTile <= ks.all_hi)) {
      // register 4 t + i is key keyv + 4 t + i
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = keyv + 4 * t + i;
            sc[r][t][i] = key >= low[r] && key < ks.hi && (bits[r] >> (4 * t + i) & 1) ? sc[r][t][i] : -INFINITY;
          }
      }
    }
    float mx[R], gap[R];
    bool move = false, far = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mx[r] = -INFINITY;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[r] = fmaxf(mx[r], sc[r][t][i]);
      mx[r] *= kscale;
      // a lane without a visible key has no say about the exponents
      gap[r] = mx[r] > -INFINITY ? own_b - e[r] : 0.0f;
      far |= fabsf(gap[r]) > kTreeGap;
      move |= mx[r] > m[r] + 8.0f;
    }
    // A row's references move where it asks for it, whatever its neighbours in the wave do: its bits do not
    // depend on theirs (in k_attn_tiles they move for all rows of a wave).
    float share[R];
#pragma unroll
    for (int r = 0; r < R; ++r) share[r] = __builtin_amdgcn_exp2f(-(gap[r] + kTreeUp));
    if (__any(move || far)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool seen = mx[r] > -INFINITY;
        const float own = ceilf(mx[r]) + own_b;
        float top = fmaxf(mx[r], __shfl_xor(mx[r], 16)), off = fabsf(gap[r]);
        top = fmaxf(top, __shfl_xor(top, 32));
        off = fmaxf(off, __shfl_xor(off, 16));
        off = fmaxf(off, __shfl_xor(off, 32));
        const bool mine = off > kTreeGap;          // (the same for the row's lanes, as all of these)
        const float mn = mine || top > m[r] + 8.0f ? fmaxf(m[r], floorf(top)) : m[r], ref = mn == -INFINITY ? 0.0f : mn;
        float fix = __builtin_amdgcn_exp2f((m[r] == -INFINITY ? mn : m[r]) - ref);
        if (m[r] == -INFINITY) fix = mn == -INFINITY ? 1.0f : 0.0f;
        l[r] *= fix;
        if constexpr (LW) l16[r] *= fix;
        if (__any(mine)) {
          // the largest weight of this tile is 2^most at most, that of the keys before 2^(m + e) to within the
          // gap; the tile's sum is taken from exponentials of its own
          float most = fmaxf(own, __shfl_xor(own, 16));
          most = fmaxf(most, __shfl_xor(most, 32));
          float sum = 0.0f;
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r][t][i], kscale, -ref));
          if (mine) {
            const float to = mn == -INFINITY ? e[r] : fmaxf(most - mn, e[r] - (mn - m[r]));
            fix = __builtin_amdgcn_exp2f(m[r] - ref + (e[r] - to));
            e[r] = to;
            gap[r] = seen ? own_b - e[r] : 0.0f;
            // (where the rounded weights count, those of pages not far below go on as they are below)
            const bool near = LW && gap[r] >= -kTreeGap;
            share[r] = near ? __builtin_amdgcn_exp2f(-(gap[r] + kTreeUp)) : 0.0f;
            l[r] += near ? 0.0f : sum;
            if constexpr (LW) l16[r] += near ? 0.0f : sum;
          }
        }
        m[r] = mn;
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] *= fix;
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float wref = (m[r] == -INFINITY ? 0.0f : m[r]) - (gap[r] + kTreeUp);
      float sum = 0.0f, sum16 = 0.0f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc[r][t][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r][t][i], kscale, -wref));
          sum += sc[r][t][i];
        }
        pf[r][t >> 1][2 * (t & 1)] = (int)pack2_out<DT_F16>(sc[r][t][0], sc[r][t][1]);
        pf[r][t >> 1][2 * (t & 1) + 1] = (int)pack2_out<DT_F16>(sc[r][t][2], sc[r][t][3]);
      }
      l[r] = __builtin_fmaf(sum, share[r], l[r]);
      if constexpr (LW) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum16 = add2(pf[r][i >> 2][i & 3], sum16);
        l16[r] = __builtin_fmaf(sum16, share[r], l16[r]);
      }
    }
  }
  __device__ __forceinline__ void finish() {       // the sums over the row's lanes
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] += __shfl_xor(l[r], 16);
      l[r] += __shfl_xor(l[r], 32);
      if constexpr (LW) {
        l16[r] += __shfl_xor(l16[r], 16);
        l16[r] += __shfl_xor(l16[r], 32);
      } else {
        l16[r] = l[r];
      }
    }
  }
  __device__ __forceinline__ bool has_nan() const {
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n) sum += (acc[r][n][0] + acc[r][n][1]) + (acc[r][n][2] + acc[r][n][3]);
    return __any(sum != sum);
  }
  __device__ __forceinline__ int unit(int r) const { return (int)(e[r] - (127.0f + kTreeUp)); }
};
// Codes of 16 keys from keyv on of a feature: those of keys that no row sees may be anything and are cleared,
// and (`careful`) NaN codes of keys that some row does not see.
__device__ __forceinline__ v4i cleared(v4i x, int keyv, const Keys& ks, bool careful) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t keep = 0, some = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = keyv + 4 * w + i;
      keep |= key >= ks.lo && key < ks.hi ? 0xffu << (8 * i) : 0u;
      some |= key < ks.all_lo || key >= ks.all_hi ? 0x80u << (8 * i) : 0u;
    }
    x[w] = (int)((uint32_t)x[w] & keep);
    if (careful) x[w] = without_nan(x[w], some);
  }
  return x;
}

// A barrier for what is in LDS: loads on their way to registers stay on it
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(kLgkmcnt0);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int D, int DT, int NW, int R, int EU>
__global__ __launch_bounds__(64 * NW, EU) void k_tree_rows(const AttnArgs a, int row_tiles, int chunk, int sorted) {
  constexpr int KL = D / 64, NT = D / 16, RB = 16 * R;
  const KvView& kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int split = blockIdx.x, head = blockIdx.y;
  int s = blockIdx.z / row_tiles;
  const int tile0 = blockIdx.z % row_tiles;
  const int group = a.heads / kv.kv_heads;
  if (sorted) {
    // the s-th longest, so that the workgroups that start last are short ones: lane l counts the sequences
    // that go before l
    const int len = lane < kv.seqs ? kv.kv_len[lane] : -1;
    int before = 0;
    for (int i = 0; i < kv.seqs; ++i) {
      const int other = __builtin_amdgcn_readlane(len, i);
      before += other > len || (other == len && i < lane) ? 1 : 0;
    }
    s = __builtin_ctzll(__ballot(lane < kv.seqs && before == s));
  }
  {
    const int q0 = kv.q_start[s], q1 = kv.q_start[s + 1], len = kv.kv_len[s];
    asm volatile("" ::"s"(q0), "s"(q1), "s"(len));             // all requested at once
  }
  const Span sp = span_of(a, s);
  const int rows = sp.n * group;
  const bool split_out = gridDim.x > 1;
  const int page_log2 = 31 - __builtin_clz(kv.page);
  const float scale = fabsf(a.scale_log2);

  __shared__ __attribute__((aligned(16))) float s_acc[NW][RB][D + 4];
  __shared__ float s_ml[NW][RB][3];
  __shared__ int s_nan[NW];
  // of each 32-key half of up to kMeta / 2 steps: page x head, and the exponent bytes (keys | values << 8)
  __shared__ int s_ph[kMeta], s_exp[kMeta];

  // keys that some row sees, and those that all do (the same for all rows of a tree)
  const Keys ks = keys_of<true>(a, sp, 0, 0);
  const int klo = ks.lo, khi = ks.hi, all_lo = ks.all_lo, all_hi = ks.all_hi;
  const bool mixed = all_lo != klo || all_hi != khi;
  // this workgroup's share: `chunk` keys from a multiple of kTile on, the last share all that is left
  const int first = klo & ~(kTile - 1);
  const int64_t from = (int64_t)split * chunk;
  const int kb0 = first + from < khi ? first + (int)from : khi;
  const int kb1 = split + 1 < (int)gridDim.x && kb0 + (int64_t)chunk < khi ? kb0 + chunk : khi;

  bool careful = false;              // the row block is taken again, without NaN codes
  for (int r0 = tile0 * RB; r0 < rows;) {
    TreeRows<D, DT, R> x;
    x.r0 = r0;
    x.rows = rows;
    x.group = group;
    x.start(a, sp, head, lr, lg);
    constexpr int kStride = NW * kTile, kRun = kMeta / 2 * kTile;
    for (int run = kb0; run < kb1; run += kRun) {
    const int stop = run + (int64_t)kRun < kb1 ? run + kRun : kb1;
    v4i kx[4][KL], vx[NT];
    // ph: page x head of the 32-key half that the lane reads
    auto request_keys = [&](int kb, auto ph) {
      int me = lane;
      asm volatile("" : "+v"(me));                 // (what follows from it need not live through the loop)
      const int row = me & 15, off = (kb + 16 * (row >> 2)) & (kv.page - 1);
      const uint8_t* const p = kv.k + ((int64_t)ph(row >> 3) * kv.page + (off + (row & 3))) * D + 16 * (me >> 4);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < KL; ++i) kx[t][i] = *(const v4i*)(p + t * 4 * D + 64 * i);
    };
    auto request_values = [&](int kb, auto ph) {
      int me = lane;
      asm volatile("" : "+v"(me));
      const int g = me >> 4, off = (kb + 16 * g) & (kv.page - 1);
      const uint8_t* const p = kv.v + ((int64_t)ph(g >> 1) * D + (me & 15)) * kv.page + off;
#pragma unroll
      for (int n = 0; n < NT; ++n) vx[n] = *(const v4i*)(p + 16 * n * kv.page);
    };

    // Every tile requests the next one, the last one itself again: with a request that may be left out the
    // compiler cannot count the loads in flight, and waits for all of them.
    int kb = run + wave * kTile;
    // Page x head of the half at `key`; one that no row sees reads page 0
    auto ph_of = [&](int key) {
      const bool seen = key < khi && key + 32 > klo;
      int p = seen ? kv.table[(int64_t)s * kv.max_pages + (key >> page_log2)] : 0;
      p = p < 0 ? 0 : (p >= kv.num_pages ? kv.num_pages - 1 : p);
      return p * kv.kv_heads + head;
    };
    // The first tiles are requested as soon as their pages are known, beside the run's exponents
    {
      constexpr int kEach = kMeta / (64 * NW);
      static_assert(kMeta % (64 * NW) == 0, "entries of a thread");
      int ph[kEach], eb[kEach];
      const int pa = ph_of(kb), pb = ph_of(kb + 32);
#pragma unroll
      for (int i = 0; i < kEach; ++i) ph[i] = ph_of(run + 32 * (tid + 64 * NW * i));
#pragma unroll
      for (int i = 0; i < kEach; ++i) eb[i] = kv.ke[ph[i]] | kv.ve[ph[i]] << 8;
      auto mine = [&](int half) { return half ? pb : pa; };
      request_keys(kb, mine);        // (a wave without a tile some others: with a branch all wait for it)
      request_values(kb, mine);
      lds_barrier();                 // the run before is read
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        s_ph[tid + 64 * NW * i] = ph[i];
        s_exp[tid + 64 * NW * i] = eb[i];
      }
      lds_barrier();
    }
    for (; kb < stop; kb += kStride) {
      const int keyv = kb + 16 * lg, exps = s_exp[((kb - run) >> 5) + (lg >> 1)];
      // (requested ahead of the keys behind this tile)
      int low[R];
      uint32_t bits[R];
      if (!(kb >= all_lo && kb + kTile <= all_hi)) {
        int me = lane;
        asm volatile("" : "+v"(me));
        x.seen(a, sp, kb, me & 15, me >> 4, low, bits);
      }
      v4f sc[R][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int r = 0; r < R; ++r) sc[r][t] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < KL; ++i) {
          const v4i lo = widen8<DT>(kx[t][i][0], kx[t][i][1], 1.0f), hi = widen8<DT>(kx[t][i][2], kx[t][i][3], 1.0f);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            sc[r][t] = mma16<DT>(lo, x.qf[r][2 * i], sc[r][t]);
            sc[r][t] = mma16<DT>(hi, x.qf[r][2 * i + 1], sc[r][t]);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      const int next = kb + kStride < stop ? kb + kStride : kb;
      auto listed = [&](int half) { return s_ph[((next - run) >> 5) + half]; };
      request_keys(next, listed);
      __builtin_amdgcn_sched_barrier(0);
      v4i pf[R][2];
      int at_lane = lane;
      asm volatile("" : "+v"(at_lane));             // (what follows from it need not live through the loop)
      x.weigh(a, sp, ks, kb, at_lane & 15, at_lane >> 4, exps, scale, low, bits, sc, pf);
      if (__builtin_expect(careful || kb < klo || kb + kTile > khi, 0)) {
        int at = keyv;
        asm volatile("" : "+v"(at));               // nothing of this ahead of the loop
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          vx[n] = cleared(vx[n], at, ks, careful);
          __builtin_amdgcn_sched_barrier(0);       // one after the other: the registers are all taken
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const v4i lo = widen8<DT_F16>(vx[n][0], vx[n][1], 1.0f), hi = widen8<DT_F16>(vx[n][2], vx[n][3], 1.0f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          x.acc[r][n] = mma16<DT_F16>(lo, pf[r][0], x.acc[r][n]);
          x.acc[r][n] = mma16<DT_F16>(hi, pf[r][1], x.acc[r][n]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      request_values(next, listed);
      __builtin_amdgcn_sched_barrier(0);
    }
    }

    // join the waves
    __syncthreads();                 // the row block before is read
    x.finish();
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int n = 0; n < NT; ++n) *(v4f*)&s_acc[wave][16 * r + lr][16 * n + 4 * lg] = scaled4(x.acc[r][n], x.unit(r));
      if (lg == 0) {
        s_ml[wave][16 * r + lr][0] = x.m[r];
        s_ml[wave][16 * r + lr][1] = x.l[r];
        s_ml[wave][16 * r + lr][2] = x.l16[r];
      }
    }
    if (mixed) {
      const int nan = x.has_nan();
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
    // 16 threads a row, each D / 16 features
    for (int at = tid >> 4; at < RB; at += 4 * NW) {
      const int orw = r0 + at, part = tid & 15;
      if (orw >= rows) break;
      float mm = s_ml[0][at][0];
#pragma unroll
      for (int w = 1; w < NW; ++w) mm = fmaxf(mm, s_ml[w][at][0]);
      const float ref = mm == -INFINITY ? 0.0f : mm;
      float f[NW], ll = 0.0f, by = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        f[w] = __builtin_amdgcn_exp2f(s_ml[w][at][0] - ref);
        ll += f[w] * s_ml[w][at][1];
        by += f[w] * s_ml[w][at][2];
      }
      const int otok = orw / group, oh = orw - otok * group;
      const int64_t orow = (int64_t)(sp.first + otok) * a.heads + head * group + oh;
      const float inv = by == 0.0f ? 0.0f : 1.0f / by;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const int d = part * 4 + c * 64;
        v4f o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < NW; ++w) o += *(const v4f*)&s_acc[w][at][d] * f[w];
        if (split_out) {
          *(v4f*)(a.part + ((int64_t)split * kv.tokens * a.heads + orow) * D + d) = o;
        } else {
          o *= inv;
          *(v2i*)((uint16_t*)a.out + orow * D + d) = v2i{(int)pack2_out<DT>(o[0], o[1]), (int)pack2_out<DT>(o[2], o[3])};
        }
      }
      if (__builtin_expect(careful, 0))
        put_nan<D, true>(a, s, head, orow, drafted_at(a, sp.first, otok, sp.past, sp.n), split, split_out, kb0, kb1, all_lo, all_hi,
                         part * 4, 64, sp.past);
      if (part == 0) {
        if (split_out) {
          float* ml = a.part_ml + ((int64_t)split * kv.tokens * a.heads + orow) * kMl<true>;
          ml[0] = mm;
          ml[1] = ll;
          ml[2] = by;
        } else if (a.lse) {
          a.lse[orow] = ll == 0.0f ? -INFINITY : (mm + __builtin_amdgcn_logf(ll)) * 0.6931471805599453f;
        }
      }
    }
    careful = false;
    r0 = rows - r0 > row_tiles * RB ? r0 + row_tiles * RB : rows;
  }
}

template <int D, int DT>
hipError_t launch_dim(const AttnArgs& a, hipStream_t st) {
  const int64_t rows = (int64_t)a.max_q * (a.heads / a.kv.kv_heads);
  const AttnPlan p = tree_plan(rows, D, a.kv.kv_heads, a.kv.seqs, a.max_q, a.max_kv, a.window);
  const int blocks = (int)p.blocks;
  if (p.per <= 32) {
    // The longest sequences first where one to four rounds of workgroups follow each other (32 sequences on 700
    // to 4100 keys, 8 kv heads of 128 features: 88 rows 72.4 -> 65.5 us, 176 rows 97 -> 91); more rounds
    // even themselves out (64 features, 176 rows, six rounds: 62.4 -> 64.9).
    const int64_t groups = (int64_t)p.splits * a.kv.kv_heads * p.blocks * a.kv.seqs;
    const int sorted = a.kv.seqs > 1 && a.kv.seqs <= 64 && a.window == 0 && groups > 512 && groups <= 2048;
    const dim3 grid((unsigned)p.splits, (unsigned)a.kv.kv_heads, (unsigned)(p.blocks * a.kv.seqs));
    if constexpr (D == 128) {
      if (p.per == 32) k_tree_rows<D, DT, 4, 2, 2><<<grid, 256, 0, st>>>(a, blocks, p.chunk, sorted);
    }
    if (p.per == 16) k_tree_rows<D, DT, 4, 1, D == 256 ? 1 : 2><<<grid, 256, 0, st>>>(a, blocks, p.chunk, sorted);
  } else {
    const unsigned grid = (unsigned)(p.blocks * a.kv.seqs * a.kv.kv_heads * p.splits);
    if constexpr (D == 256) k_attn_tiles<D, DT, 4, true><<<grid, 256, 0, st>>>(a, blocks, p.splits, p.chunk);
    else k_attn_tiles<D, DT, 8, true><<<grid, 512, 0, st>>>(a, blocks, p.splits, p.chunk);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t jb = join_blocks(a.max_q, a.heads, a.kv.seqs);
  k_attn_join<D, DT, true><<<(unsigned)(jb * a.kv.seqs), 256, 0, st>>>(a, (int)jb, p.splits);
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

int tree_splits(int heads, int kv_heads, int dim, int seqs, int64_t max_q, int64_t max_kv, int window) {
  return tree_plan(max_q * (heads / kv_heads), dim, kv_heads, seqs, max_q, max_kv, window).splits;
}

hipError_t launch_attention_tree(const AttnArgs& a, int dt, int dim, hipStream_t st) {
  return dt == DT_F16 ? launch_dt<DT_F16>(a, dim, st) : launch_dt<DT_BF16>(a, dim, st);
}

}  // namespace q8
