// The append with each head of the new keys and queries normalised before it is
// rotated, and positions of the tokens' own (drafted trees).
//
// Work is cut by page as in kv_append.hip.  A thread of the keys takes P tokens x
// 16 features, the two groups of 8 that the rotation pairs (or neighbours), so
// that D / 16 neighbouring lanes hold a head: the mean square is a sum over them,
// a partner's feature is in the same thread, and the finished values wait in
// registers for the page's maximum.  A thread of the values takes 8 tokens x 8
// features, kept as they were read.  Everything is read once.
//
// 15372 new tokens of 6 prompts (32 query and 8 kv heads of 128 features, f16, pages of 128, 64 features turned as
// neighbours): 82 us, 350 MB at 4.3 TB/s where a large copy moves 5.2.  Keys and values alone take 29, queries alone at
// the copy's rate would take 44.  A head's groups of 8 lie beside each other over the threads (u and u + dim / 16), so
// that requests of neighbouring lanes fill whole lines (with 32 bytes a thread in a row 102 us for 97, then); what
// follows from a lane's place is computed in the loops, or it is spilled ahead of them, 100 MB of stores (97 for 82).
// 12 drafts or 128 single tokens: 6 us, a chain of length, page, exponent and codes.
// Heads of 256 features on pages of 128 have four tokens a thread and spill 80 to 90 registers: the same prompts as
// bf16 on 16 over 4 such heads 107 us, 85 on pages of 64, floor 71; 12 drafts 10 us.  Input of 32 bits (32 over 8 heads of
// 128, 7684 tokens) 78 us where its bytes take 67, of 16 bits 36 (floor 35).
#include "q8_kv_append.hpp"

namespace q8 {
namespace {

// Features x_i become (x_i r) w_i, each product rounded, r = 1 / sqrt(mean x^2 + eps) rounded to binary32
// from a sum in binary64 (the squares of 16-bit values are exact there, so that the order of the lanes does
// not matter).
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// over N neighbouring lanes (4, 8 or 16), which all run this together
template <int N>
__device__ __forceinline__ double lanes_sum(double v) {
  static_assert(N == 4 || N == 8 || N == 16, "lanes of a head");
  v += dpp_f64<0xB1>(v);
  v += dpp_f64<0x4E>(v);
  if constexpr (N >= 8) v += dpp_f64<0x141>(v);
  if constexpr (N >= 16) v += dpp_f64<0x140>(v);
  return v;
}
__device__ __forceinline__ double squares8(const float* v, double sum) {
#pragma unroll
  for (int e = 0; e < 8; ++e) sum = __builtin_fma((double)v[e], (double)v[e], sum);
  return sum;
}
// 1 / sqrt(m): the hardware's t (some 23 bits) times (1 - e)^(-1/2) = 1 + e / 2 + 3 e^2 / 8 + ..., e = 1 - m t^2;
// 0 for an infinite m, where that is NaN
__device__ __forceinline__ float inverse_root(double m) {
  const double t = __builtin_amdgcn_rsq(m);
  const double e = __builtin_fma(-(m * t), t, 1.0);
  return (float)(m < __builtin_huge_val() ? __builtin_fma(t * e, __builtin_fma(e, 0.375, 0.5), t) : t);
}
__device__ __forceinline__ void load_weight(const AppendArgs& a, const void* w, int c, float* v) {
  if (w == nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.0f;
  } else if (a.w_dt == DT_F32) {
    load8<DT_F32>(w, 8 * c, v);
  } else if (a.w_dt == DT_F16) {
    load8<DT_F16>(w, 8 * c, v);
  } else {
    load8<DT_BF16>(w, 8 * c, v);
  }
}
// The position that a token is rotated by: its own where positions are given, else that of its slot.
__device__ __forceinline__ int turned_by(const AppendArgs& a, int token, int slot) {
  const int p = a.pos ? a.pos[token] : slot;
  return p < 0 ? 0 : p;
}
// The two groups of 8 features of thread u of a head, and whether they are turned: where the rotation leaves
// the choice, neighbouring threads have neighbouring groups.
struct Groups {
  int c0, c1;
  bool t0, t1;
};
template <int D>
__device__ __forceinline__ Groups groups_of(const AppendArgs& a, int u) {
  const int pairs = a.rot >> 4;
  if (a.interleaved || a.rot == 0) return Groups{u, u + D / 16, u < 2 * pairs, u + D / 16 < 2 * pairs};
  return u < pairs ? Groups{u, u + pairs, true, true} : Groups{2 * u, 2 * u + 1, false, false};
}
// Their cosines and sines at a position, of four pairs each where pairs are neighbours (2 i, 2 i + 1), else
// those of pairs 8u .. 8u+7.  Threads whose features are not turned read others' and leave them.
__device__ __forceinline__ void load_angles(const AppendArgs& a, const Groups& g, int u, int pos, float* co, float* si) {
  const int64_t row = (int64_t)(pos < a.positions ? pos : a.positions - 1) * (a.rot >> 1);
  const int o0 = g.t0 ? (a.interleaved ? 4 * g.c0 : 8 * u) : 0, o1 = a.interleaved ? (g.t1 ? 4 * g.c1 : 0) : o0 + 4;
  *(v4f*)co = *(const v4f*)(a.cos + row + o0);
  *(v4f*)(co + 4) = *(const v4f*)(a.cos + row + o1);
  *(v4f*)si = *(const v4f*)(a.sin + row + o0);
  *(v4f*)(si + 4) = *(const v4f*)(a.sin + row + o1);
}
// A head's 16 features of this thread normalised (weights given) and turned
template <int D>
__device__ __forceinline__ void finish16(const AppendArgs& a, const Groups& g, bool norm, const float* w0, const float* w1,
                                         const float* co, const float* si, float* v, float* w) {
  if (norm) {
    const float r = inverse_root(lanes_sum<D / 16>(squares8(w, squares8(v, 0.0))) * (1.0 / D) + (double)a.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = v[e] * r * w0[e];
      w[e] = w[e] * r * w1[e];
    }
  }
  if (a.rot == 0 || !g.t0) return;                 // (the second group is turned only where the first is)
  {
#pragma clang fp contract(off)
    if (a.interleaved) {                                     // uniform
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = v[2 * i], q = v[2 * i + 1];
        v[2 * i] = p * co[i] - q * si[i];
        v[2 * i + 1] = q * co[i] + p * si[i];
      }
      if (g.t1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float r = w[2 * i], s = w[2 * i + 1];
          w[2 * i] = r * co[4 + i] - s * si[4 + i];
          w[2 * i + 1] = s * co[4 + i] + r * si[4 + i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = v[i], q = w[i];
        v[i] = p * co[i] - q * si[i];
        w[i] = q * co[i] + p * si[i];
      }
    }
  }
}

template <int DT, int D, int B>
struct Shape {
  static constexpr int kUnits = D / 16;                          // threads of a head
  static constexpr int kTokens = B * D > 128 * 128 ? 4 : 2;      // of a thread of the keys
  static constexpr int kKeys = B / kTokens * kUnits;             // threads of a page and head: of its keys,
  static constexpr int kVals = B / 8 * (D / 8);                  // and of its values
  static constexpr int kThreads = kKeys > 256 ? kKeys : 256;
  static constexpr int kKeyItems = kThreads / (kKeys > 64 ? kKeys : 64), kValItems = kThreads / (kVals > 64 ? kVals : 64);
  static_assert(kThreads <= 512 && kVals <= kThreads && kThreads % (kVals > 64 ? kVals : 64) == 0, "items of a workgroup");
};

// The largest of an item's values: WAVES neighbouring waves hold it (all of the workgroup's run this)
template <int WAVES>
__device__ __forceinline__ float item_max(float v, float* red) {
  v = wave_max(v);
  if constexpr (WAVES > 1) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v = fmaxf(v, red[wave / WAVES * WAVES + w]);
  }
  return v;
}

// A lane's place, so that what follows from it is computed in the loop (which most threads run once) and not
// kept in registers ahead of it
__device__ __forceinline__ int in_loop(int place) {
  asm volatile("" : "+v"(place));
  return place;
}

// The slots of a sequence's new tokens
struct Slots {
  int first, past, lo, hi;
};
template <int B>
__device__ __forceinline__ Slots slots_of(const KvView& kv, int s) {
  Slots r;
  int end = kv.q_start[s + 1], first = kv.q_start[s];
  end = end < 0 ? 0 : (end > kv.tokens ? kv.tokens : end);
  first = first < 0 ? 0 : (first > end ? end : first);
  const int len = kv.kv_len[s], total = len < 0 ? 0 : len;
  const int64_t cap = (int64_t)kv.max_pages * B;
  r.first = first;
  r.past = total - (end - first);
  r.lo = r.past < 0 ? 0 : r.past;
  r.hi = total < cap ? total : (int)cap;
  return r;
}

__device__ __forceinline__ void codes8(const float* v, int b, uint32_t& q0, uint32_t& q1) {
  float u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = __builtin_ldexpf(v[e], 127 - b);
  q0 = pack4_e4m3(u[0], u[1], u[2], u[3]);
  q1 = pack4_e4m3(u[4], u[5], u[6], u[7]);
}

template <int DT, int D, int B>
__device__ __forceinline__ void append_keys(const AppendArgs& a, int s, int j0, int group, float* red) {
  using SH = Shape<DT, D, B>;
  constexpr int P = SH::kTokens, U = SH::kUnits, WAVES = SH::kKeys > 64 ? SH::kKeys / 64 : 1;
  const KvView& kv = a.kv;
  const Slots sl = slots_of<B>(kv, s);
  if (sl.lo >= sl.hi) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int head = group * SH::kKeyItems + wave / WAVES;
  const int last = (sl.hi - 1) / B;
  for (int lp = sl.lo / B + j0; lp <= last; lp += a.reach) {
    const int in_item = in_loop((wave % WAVES) * 64 + (threadIdx.x & 63));
    const bool have = head < kv.kv_heads && in_item < SH::kKeys;
    const int u = in_item % U, tg = in_item / U;
    const Groups g = groups_of<D>(a, u);
    float w0[8], w1[8];
    load_weight(a, a.kw, g.c0, w0);
    load_weight(a, a.kw, g.c1, w1);
    const int page = kv.table[(int64_t)s * kv.max_pages + lp];
    const bool here = page >= 0 && page < kv.num_pages;
    const int64_t ph = (int64_t)(here ? page : 0) * kv.kv_heads + (have ? head : 0);
    const int had = kv.ke[ph];
    // this thread's slots: new ones [i0, i1) of P
    const int base = lp * B + P * tg;
    int i0 = sl.lo - base, i1 = sl.hi - base;
    i0 = i0 < 0 ? 0 : (i0 > P ? P : i0);
    i1 = i1 < 0 ? 0 : (i1 > P ? P : i1);
    if (!have) i0 = i1 = 0;
    float v[P][8], w[P][8], amax = 0.0f;
    if (i0 < i1) {                   // (the same for all lanes of a head)
      float co[P][8], si[P][8];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        // places without a new token repeat one that is
        const int k = i < i0 ? i0 : (i < i1 ? i : i1 - 1), token = sl.first + (base + k - sl.past);
        const int64_t off = (int64_t)token * a.k_stride + (int64_t)head * D;
        load8<DT>(a.k, off + 8 * g.c0, v[i]);
        load8<DT>(a.k, off + 8 * g.c1, w[i]);
        if (a.rot) load_angles(a, g, u, turned_by(a, token, base + k), co[i], si[i]);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        finish16<D>(a, g, a.kw != nullptr, w0, w1, co[i], si[i], v[i], w[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(v[i][e]), fabsf(w[i][e])));
      }
    }
    amax = item_max<WAVES>(amax, red);
    if (!have || !here) continue;
    const bool fresh = sl.lo <= lp * B;            // no token of the page is older than this call's
    const int want = exponent_byte(amax), b = fresh ? want : (had > want ? had : want);
    const int shift = fresh ? 0 : had - b;
    if (in_item == 0 && b != had) kv.ke[ph] = (uint8_t)b;
    uint8_t* const rows = kv.k + ph * (D * B) + (int64_t)(P * tg) * D;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      v2i* const p0 = (v2i*)(rows + i * D + 8 * g.c0);
      v2i* const p1 = (v2i*)(rows + i * D + 8 * g.c1);
      if (i >= i0 && i < i1) {
        uint32_t q0, q1;
        codes8(v[i], b, q0, q1);
        *p0 = v2i{(int)q0, (int)q1};
        codes8(w[i], b, q0, q1);
        *p1 = v2i{(int)q0, (int)q1};
      } else if (shift < 0 && base + i < sl.lo) {              // an older token at the new scale
        const v2i x = *p0, y = *p1;
        *p0 = v2i{(int)rescale4((uint32_t)x[0], shift), (int)rescale4((uint32_t)x[1], shift)};
        *p1 = v2i{(int)rescale4((uint32_t)y[0], shift), (int)rescale4((uint32_t)y[1], shift)};
      }
    }
  }
}

template <int DT, int D, int B>
__device__ __forceinline__ void append_values(const AppendArgs& a, int s, int j0, int group, float* red) {
  using SH = Shape<DT, D, B>;
  constexpr int C = D / 8, WAVES = SH::kVals > 64 ? SH::kVals / 64 : 1;
  const KvView& kv = a.kv;
  const Slots sl = slots_of<B>(kv, s);
  if (sl.lo >= sl.hi) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int head = group * SH::kValItems + wave / WAVES;
  const int last = (sl.hi - 1) / B;
  for (int lp = sl.lo / B + j0; lp <= last; lp += a.reach) {
    const int in_item = in_loop((wave % WAVES) * 64 + (threadIdx.x & 63));
    const bool have = head < kv.kv_heads && in_item < SH::kVals;
    const int c = in_item % C, tg = in_item / C;
    const int page = kv.table[(int64_t)s * kv.max_pages + lp];
    const bool here = page >= 0 && page < kv.num_pages;
    const int64_t ph = (int64_t)(here ? page : 0) * kv.kv_heads + (have ? head : 0);
    const int had = kv.ve[ph];
    const int base = lp * B + 8 * tg;
    int i0 = sl.lo - base, i1 = sl.hi - base;
    i0 = i0 < 0 ? 0 : (i0 > 8 ? 8 : i0);
    i1 = i1 < 0 ? 0 : (i1 > 8 ? 8 : i1);
    if (!have) i0 = i1 = 0;
    constexpr int R = DT == DT_F32 ? 2 : 1;        // 16-byte pieces of 8 features
    v4i raw[8][R];
    float amax = 0.0f;
    auto values = [&](int i, float* v) {
#pragma unroll
      for (int r = 0; r < R; ++r) Chunk<DT>::decode(raw[i][r], v + r * Chunk<DT>::kElems);
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int r = 0; r < R; ++r) raw[i][r] = v4i{0, 0, 0, 0};
      if (i < i0 || i >= i1) continue;
      const int64_t off = (int64_t)(sl.first + (base + i - sl.past)) * a.v_stride + (int64_t)head * D + 8 * c;
      const v4i* const p = DT == DT_F32 ? (const v4i*)((const float*)a.v + off) : (const v4i*)((const uint16_t*)a.v + off);
#pragma unroll
      for (int r = 0; r < R; ++r) raw[i][r] = p[r];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      values(i, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
    }
    amax = item_max<WAVES>(amax, red);
    if (!have || !here) continue;
    const bool fresh = sl.lo <= lp * B;
    const int want = exponent_byte(amax), b = fresh ? want : (had > want ? had : want);
    const int shift = fresh ? 0 : had - b;
    if (in_item == 0 && b != had) kv.ve[ph] = (uint8_t)b;
    const int old = shift < 0 ? (sl.lo - base < 0 ? 0 : (sl.lo - base > 8 ? 8 : sl.lo - base)) : 0;
    if (i0 >= i1 && old == 0) continue;
    // the tokens of a feature together: 4 x 4 byte transpositions
    uint32_t o[8][2];                              // [feature][four tokens]
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t q[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[8];
        values(4 * x + j, v);
        codes8(v, b, q[j][0], q[j][1]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t l01 = __builtin_amdgcn_perm(q[1][h], q[0][h], 0x05010400u), h01 = __builtin_amdgcn_perm(q[1][h], q[0][h], 0x07030602u);
        const uint32_t l23 = __builtin_amdgcn_perm(q[3][h], q[2][h], 0x05010400u), h23 = __builtin_amdgcn_perm(q[3][h], q[2][h], 0x07030602u);
        o[4 * h][x] = __builtin_amdgcn_perm(l23, l01, 0x05040100u);
        o[4 * h + 1][x] = __builtin_amdgcn_perm(l23, l01, 0x07060302u);
        o[4 * h + 2][x] = __builtin_amdgcn_perm(h23, h01, 0x05040100u);
        o[4 * h + 3][x] = __builtin_amdgcn_perm(h23, h01, 0x07060302u);
      }
    }
    uint8_t* const rows = kv.v + ph * (D * B) + (int64_t)(8 * c) * B + 8 * tg;
    if (i0 > 0 || i1 < 8) {
      // bytes of older tokens stay, at the new scale, and so do those behind (the 8 x 8 are this thread's alone)
      uint32_t put[2], was[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        put[x] = was[x] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          put[x] |= 4 * x + j >= i0 && 4 * x + j < i1 ? 0xffu << (8 * j) : 0u;
          was[x] |= 4 * x + j < old ? 0xffu << (8 * j) : 0u;
        }
      }
      v2i y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = *(const v2i*)(rows + e * B);
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t z = (uint32_t)y[e][x];
          if (old > 0) z = (rescale4(z, shift) & was[x]) | (z & ~was[x]);
          o[e][x] = (o[e][x] & put[x]) | (z & ~put[x]);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) *(v2i*)(rows + e * B) = v2i{(int)o[e][0], (int)o[e][1]};
  }
}

// One new token of a sequence: D / 16 lanes hold a kv head's keys or values, 16 features each (u: which),
// and decide its scale among themselves.
template <int DT, int D, int B, bool V>
__device__ __forceinline__ void append_head(const AppendArgs& a, int s, int first, int pos, int head, int u) {
  constexpr int U = D / 16;
  const KvView& kv = a.kv;
  const int lp = pos / B, off = pos % B;
  const int page = lp < kv.max_pages ? kv.table[(int64_t)s * kv.max_pages + lp] : -1;
  const bool have = head < kv.kv_heads, here = page >= 0 && page < kv.num_pages;
  head = have ? head : 0;
  const int64_t ph = (int64_t)(here ? page : 0) * kv.kv_heads + head;
  uint8_t* const exps = (V ? kv.ve : kv.ke) + ph;
  const int had = *exps;
  const Groups g = V ? Groups{u, u + U, false, false} : groups_of<D>(a, u);
  const void* const x = V ? a.v : a.k;
  const int64_t from = (int64_t)first * (V ? a.v_stride : a.k_stride) + (int64_t)head * D;
  float v[8], w[8];
  load8<DT>(x, from + 8 * g.c0, v);
  load8<DT>(x, from + 8 * g.c1, w);
  if constexpr (!V) {
    float w0[8], w1[8], co[8], si[8];
    load_weight(a, a.kw, g.c0, w0);
    load_weight(a, a.kw, g.c1, w1);
    if (a.rot) load_angles(a, g, u, turned_by(a, first, pos), co, si);
    finish16<D>(a, g, a.kw != nullptr, w0, w1, co, si, v, w);
  }
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(v[e]), fabsf(w[e])));
  // over the head's 4, 8 or 16 lanes (bit patterns of non-negative floats order as integers)
  int am = __float_as_int(amax);
  auto up = [](int x, int y) { return x > y ? x : y; };
  am = up(am, __builtin_amdgcn_update_dpp(0, am, 0xB1, 0xF, 0xF, false));
  am = up(am, __builtin_amdgcn_update_dpp(0, am, 0x4E, 0xF, 0xF, false));
  if constexpr (U >= 8) am = up(am, __builtin_amdgcn_update_dpp(0, am, 0x141, 0xF, 0xF, false));
  if constexpr (U >= 16) am = up(am, __builtin_amdgcn_update_dpp(0, am, 0x140, 0xF, 0xF, false));
  if (!have || !here) return;
  const bool fresh = off == 0;
  const int want = exponent_byte(__int_as_float(am));
  const int b = fresh ? want : (had > want ? had : want);
  const int shift = fresh ? 0 : had - b;
  if (u == 0 && b != had) *exps = (uint8_t)b;
  auto put = [&](const float* x, int c) {
    uint32_t q0, q1;
    codes8(x, b, q0, q1);
    if constexpr (!V) {
      uint8_t* const codes = kv.k + ph * (D * B) + 8 * c;
      if (shift < 0)
#pragma unroll 8
        for (int i = 0; i < off; ++i) {
          v2i* p = (v2i*)(codes + i * D);
          const v2i o = *p;
          *p = v2i{(int)rescale4((uint32_t)o[0], shift), (int)rescale4((uint32_t)o[1], shift)};
        }
      *(v2i*)(codes + off * D) = v2i{(int)q0, (int)q1};
    } else {
      uint8_t* const codes = kv.v + ph * (D * B) + (int64_t)(8 * c) * B;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint8_t* const row = codes + e * B;
        if (shift < 0)
          for (int i = 0; i < off; i += 4) {
            uint32_t* p = (uint32_t*)(row + i);
            const uint32_t mask = off - i >= 4 ? 0xffffffffu : (1u << (8 * (off - i))) - 1u;
            *p = (rescale4(*p, shift) & mask) | (*p & ~mask);
          }
        row[off] = (uint8_t)((e < 4 ? q0 : q1) >> (8 * (e & 3)));
      }
    }
  };
  put(v, g.c0);
  put(w, g.c1);
}

// The queries of one sequence: a token's 16 features of `span` heads a thread, which share their angles.
template <int DT, int D>
__device__ __forceinline__ void norm_queries(const AppendArgs& a, int s, int block, int blocks, int span, int threads) {
  constexpr int U = D / 16;                                  // threads of a head
  const KvView& kv = a.kv;
  int end = kv.q_start[s + 1], first = kv.q_start[s];
  end = end < 0 ? 0 : (end > kv.tokens ? kv.tokens : end);
  first = first < 0 ? 0 : (first > end ? end : first);
  const int len = kv.kv_len[s], past = (len < 0 ? 0 : len) - (end - first);
  const int spans = (a.heads + span - 1) / span, per = U * spans;
  const int64_t all = (int64_t)(end - first) * per;
  float w0[8], w1[8];
  {
    const Groups g = groups_of<D>(a, threadIdx.x % U);       // (blocks of threads are whole heads)
    load_weight(a, a.qw, g.c0, w0);
    load_weight(a, a.qw, g.c1, w1);
  }
  for (int64_t i = (int64_t)block * threads + threadIdx.x; i < all; i += (int64_t)blocks * threads) {
    const int t = (int)(i / per), h0 = (int)(i - (int64_t)t * per) / U * span;
    const int u = in_loop(threadIdx.x) % U;
    const Groups g = groups_of<D>(a, u);
    float co[8], si[8];
    if (a.rot) load_angles(a, g, u, turned_by(a, first + t, past + t), co, si);
    const int64_t from = (int64_t)(first + t) * a.q_stride, to = (int64_t)(first + t) * a.heads * D;
    const int h1 = h0 + span < a.heads ? h0 + span : a.heads;
    // two heads at once (the last of an odd number twice)
    for (int h = h0; h < h1; h += 2) {
      const int64_t h2 = h + 1 < h1 ? h + 1 : h;
      float v[2][8], w[2][8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t at = from + (i == 0 ? h : h2) * D;
        load8<DT>(a.q, at + 8 * g.c0, v[i]);
        load8<DT>(a.q, at + 8 * g.c1, w[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        finish16<D>(a, g, a.qw != nullptr, w0, w1, co, si, v[i], w[i]);
        const int64_t at = to + (i == 0 ? h : h2) * D;
        store8<DT>(a.q_out, at + 8 * g.c0, v[i]);
        store8<DT>(a.q_out, at + 8 * g.c1, w[i]);
      }
    }
  }
}

template <int DT, int D, int B>
__global__ __launch_bounds__((Shape<DT, D, B>::kThreads), 4) void k_kv_append_norm(const AppendArgs a, int kv_blocks, int groups,
                                                                                             int key_groups, int q_blocks, int span,
                                                                                             int token_blocks) {
  using SH = Shape<DT, D, B>;
  __shared__ float red[SH::kThreads / 64];
  // the pages' workgroups spread evenly among the queries' (kv_append.hip)
  const int64_t all = gridDim.x, i = blockIdx.x;
  const int before = (int)(i * kv_blocks / all), after = (int)((i + 1) * kv_blocks / all);
  if (after > before) {
    int s, j0 = 0, group, step = groups;
    if (token_blocks > 0) {
      // one new token a sequence is expected; a sequence with another number takes its pages here too
      s = before / token_blocks;
      group = before % token_blocks;
      step = token_blocks;
      int end = a.kv.q_start[s + 1], first = a.kv.q_start[s];
      end = end < 0 ? 0 : (end > a.kv.tokens ? a.kv.tokens : end);
      first = first < 0 ? 0 : (first > end ? end : first);
      const int pos = a.kv.kv_len[s] - 1;
      if (end - first == 1) {
        const int slot = group * SH::kThreads + threadIdx.x, head = slot / SH::kUnits, u = slot % SH::kUnits;
        if (pos < 0) return;
        if (head < a.kv.kv_heads) append_head<DT, D, B, false>(a, s, first, pos, head, u);
        else append_head<DT, D, B, true>(a, s, first, pos, head - a.kv.kv_heads, u);
        return;
      }
    } else {
      const int b = before / groups;
      s = b / a.reach;
      j0 = b % a.reach;
      group = before % groups;
    }
    for (; group < groups; group += step) {
      if (group < key_groups) append_keys<DT, D, B>(a, s, j0, group, red);
      else append_values<DT, D, B>(a, s, j0, group - key_groups, red);
    }
  } else {
    const int b = (int)i - before;
    norm_queries<DT, D>(a, b / q_blocks, b % q_blocks, q_blocks, span, SH::kThreads);
  }
}

template <int DT, int D, int B>
hipError_t launch_shape(const AppendArgs& a, hipStream_t st) {
  using SH = Shape<DT, D, B>;
  const int key_groups = (a.kv.kv_heads + SH::kKeyItems - 1) / SH::kKeyItems;
  const int groups = key_groups + (a.kv.kv_heads + SH::kValItems - 1) / SH::kValItems;
  const AppendPlan p = append_plan(a.kv.seqs, a.max_q, a.kv.max_pages, B, a.kv.kv_heads, D, a.heads, a.q ? D / 16 : 0, 0,
                                   SH::kThreads, groups, 16);
  AppendArgs part = a;
  part.reach = (int)p.reach;
  for (int s = 0; s < a.kv.seqs; s += p.seqs) {
    part.kv.seqs = a.kv.seqs - s < p.seqs ? a.kv.seqs - s : p.seqs;
    part.kv.q_start = a.kv.q_start + s;
    part.kv.kv_len = a.kv.kv_len + s;
    part.kv.table = a.kv.table + (int64_t)s * a.kv.max_pages;
    const int64_t kv_blocks = p.kv_blocks(part.kv.seqs);
    k_kv_append_norm<DT, D, B><<<(unsigned)(kv_blocks + p.q_blocks * part.kv.seqs), SH::kThreads, 0, st>>>(
        part, (int)kv_blocks, groups, key_groups, p.q_blocks > 0 ? (int)p.q_blocks : 1, p.span, (int)p.token_blocks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int D>
hipError_t launch_dim(const AppendArgs& a, hipStream_t st) {
  switch (a.kv.page) {
    case 32: return launch_shape<DT, D, 32>(a, st);
    case 64: return launch_shape<DT, D, 64>(a, st);
    default: return launch_shape<DT, D, 128>(a, st);
  }
}
template <int DT>
hipError_t launch_dt(const AppendArgs& a, int dim, hipStream_t st) {
  switch (dim) {
    case 64: return launch_dim<DT, 64>(a, st);
    case 128: return launch_dim<DT, 128>(a, st);
    default: return launch_dim<DT, 256>(a, st);
  }
}

}  // namespace

hipError_t launch_kv_append_norm(const AppendArgs& a, int dt, int dim, hipStream_t st) {
  switch (dt) {
    case DT_F32: return launch_dt<DT_F32>(a, dim, st);
    case DT_F16: return launch_dt<DT_F16>(a, dim, st);
    default: return launch_dt<DT_BF16>(a, dim, st);
  }
}

}  // namespace q8
