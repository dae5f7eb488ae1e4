// Append to the paged 8-bit key/value cache: rotate the new keys by their
// position, find each touched (page, head)'s power-of-two scale, store e4m3
// codes, and rotate the queries of the same tokens.
//
// Work is cut by page: one (sequence, touched page, kv head, K or V) is one
// item, so the scale of a page and head is decided in one place, without
// atomics, whatever the number of new tokens in it.  An item's tokens x
// features are patches of 8 tokens x 8 features, one per thread: a token's
// 8 features are one 16-byte load, K goes out as 8 bytes per token, and V,
// stored with the tokens innermost, as 8 bytes per feature, with no
// transposition through LDS.  (Patches of 16 tokens: half the waves, each
// with twice the round trips, 110 against 105 us for the keys and values of
// 15 thousand tokens beside their queries.)
//
// Bound by bytes for prompts (350 MB, 105 us, 3.3 TB/s: the queries' copy runs
// at a copy's rate, the keys and values wait for each page's maximum before the
// first code leaves) and by latency for single tokens (3.8 us of kernel for one
// sequence, 6.4 for 128, where no page's scale grows).
#include "q8_device.hpp"
#include "q8_kv.hpp"
#include "q8_kv_plan.hpp"

namespace q8 {
namespace {

constexpr int kPatch = 8;         // tokens of a patch

// 8 consecutive elements as floats
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t off, float* v) {
  if constexpr (DT == DT_F32) {
    const v4i* p = (const v4i*)((const float*)base + off);
    Chunk<DT>::decode(p[0], v);
    Chunk<DT>::decode(p[1], v + 4);
  } else {
    Chunk<DT>::decode(*(const v4i*)((const uint16_t*)base + off), v);
  }
}
template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t off, const float* v) {
  if constexpr (DT == DT_F32) {
    v4f* p = (v4f*)((float*)base + off);
    p[0] = v4f{v[0], v[1], v[2], v[3]};
    p[1] = v4f{v[4], v[5], v[6], v[7]};
  } else {
    v4i o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (int)pack2_out<DT>(v[2 * i], v[2 * i + 1]);
    *(v4i*)((uint16_t*)base + off) = o;
  }
}

// cos and sin of the 8 features 8c .. 8c+7 of a head at a position, as their rotation uses them:
// 8 of each for pairs (i, i + r), 4 of each for pairs (2 i, 2 i + 1).
struct Turn {
  float co[8], si[8];
};
__device__ __forceinline__ void load_turn(const AppendArgs& a, int c, int pos, Turn& t) {
  const int half = a.rot >> 1;
  const int64_t row = (int64_t)(pos < a.positions ? pos : a.positions - 1) * half;
  if (a.interleaved) {
    Chunk<DT_F32>::decode(*(const v4i*)(a.cos + row + 4 * c), t.co);
    Chunk<DT_F32>::decode(*(const v4i*)(a.sin + row + 4 * c), t.si);
  } else {
    const int j = 8 * c < half ? 8 * c : 8 * c - half;
    load8<DT_F32>(a.cos, row + j, t.co);
    load8<DT_F32>(a.sin, row + j, t.si);
  }
}
// Every product and the sum are rounded on their own (no contraction), so the codes do not depend on
// how the compiler pairs them.  w: the partner features (pairs (i, i + r) only), low: v is the first
// of the two.
__device__ __forceinline__ void turn8(const Turn& t, bool interleaved, bool low, float* v, const float* w) {
#pragma clang fp contract(off)
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = v[2 * i], r = v[2 * i + 1];
      v[2 * i] = p * t.co[i] - r * t.si[i];
      v[2 * i + 1] = r * t.co[i] + p * t.si[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float side = low ? -w[i] : w[i];
      v[i] = v[i] * t.co[i] + side * t.si[i];      // (a cos - b sin: the negated product rounds alike)
    }
  }
}
// The features 8c .. 8c+7 of the head at element offset `off`, rotated.  Lanes whose features are not
// rotated load the angles of others and leave them unused: a branch here makes the loads of several
// tokens wait for one another.
template <int DT>
__device__ __forceinline__ void load_rotated(const AppendArgs& a, const void* x, int64_t off, int c, int pos, float* v) {
  load8<DT>(x, off + 8 * c, v);
  if (a.rot == 0) return;                                    // uniform
  const int half = a.rot >> 1;
  const bool turned = 8 * c < a.rot, low = 8 * c < half;
  const int ct = turned ? c : 0;
  Turn t;
  float w[8] = {}, u[8];
  if (!a.interleaved) load8<DT>(x, off + (turned ? (low ? 8 * c + half : 8 * c - half) : 0), w);
  load_turn(a, ct, pos, t);
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = v[e];
  turn8(t, a.interleaved, low, u, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = turned ? u[e] : v[e];
}

// The exponent byte of a page and head: the least b with amax <= 448 2^(b - 127).
__device__ __forceinline__ int exponent_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return b < 0 ? 0 : (b > 254 ? 254 : b);
}

// Four codes re-expressed at a scale 2^-shift times as fine
__device__ __forceinline__ uint32_t rescale4(uint32_t w, int shift) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return pack4_e4m3(__builtin_ldexpf(lo[0], shift), __builtin_ldexpf(lo[1], shift), __builtin_ldexpf(hi[0], shift),
                    __builtin_ldexpf(hi[1], shift));
}

template <int DT, int D, int B>
struct Shape {
  static constexpr int kCols = D / 8;                            // 8-feature chunks of a head
  static constexpr int kPatches = (B / kPatch) * kCols;          // of one item
  static constexpr int kThreads = kPatches > 256 ? kPatches : 256;
  static constexpr int kItemWaves = kPatches > 64 ? kPatches / 64 : 1;
  static constexpr int kItems = kThreads / 64 / kItemWaves;      // items of one workgroup
};

template <int DT, int D, int B>
__device__ void append_pages(const AppendArgs& a, int s, int j0, int group, float* red) {
  using SH = Shape<DT, D, B>;
  const KvView& kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int end = kv.q_start[s + 1], first = kv.q_start[s];
  end = end < 0 ? 0 : (end > kv.tokens ? kv.tokens : end);
  first = first < 0 ? 0 : (first > end ? end : first);
  const int len = kv.kv_len[s], total = len < 0 ? 0 : len, past = total - (end - first);
  const int64_t cap = (int64_t)kv.max_pages * B;
  const int lo = past < 0 ? 0 : past, hi = total < cap ? total : (int)cap;
  if (lo >= hi) return;
  const int item = group * SH::kItems + wave / SH::kItemWaves;
  const bool is_v = item >= kv.kv_heads, have = item < 2 * kv.kv_heads;
  const int head = is_v ? item - kv.kv_heads : item;
  const int patch = (wave % SH::kItemWaves) * 64 + lane;
  const int c = patch % SH::kCols, tg = patch / SH::kCols;
  const void* const x = is_v ? a.v : a.k;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const int last = (hi - 1) / B;
  for (int lp = lo / B + j0; lp <= last; lp += a.reach) {
    // the page and the scale that it has are on their way while the new values are read
    const int page = kv.table[(int64_t)s * kv.max_pages + lp];
    const bool here = page >= 0 && page < kv.num_pages;
    const int64_t ph = (int64_t)(here ? page : 0) * kv.kv_heads + (have ? head : 0);
    uint8_t* const exps = (is_v ? kv.ve : kv.ke) + ph;
    const int had = *exps;
    const int base = lp * B + kPatch * tg;
    int i0 = lo - base, i1 = hi - base;
    i0 = i0 < 0 ? 0 : (i0 > kPatch ? kPatch : i0);
    i1 = i1 < 0 ? 0 : (i1 > kPatch ? kPatch : i1);
    const bool active = have && patch < SH::kPatches;
    if (!active) i0 = i1 = 0;
    auto row = [&](int i) { return (int64_t)(first + (base + i - past)) * stride + (int64_t)head * D; };
    // more than two new tokens in the patch: four at once (places without a new token repeat one that
    // is, and are not stored); one or two, as in decoding: one after the other
    const bool many = i1 - i0 > 2;
    float amax = 0.0f;
    // Read once for the maximum and once more (from the caches) for the codes: kept in registers instead,
    // they leave too few waves for the queries' copy in the same launch.
    auto four = [&](int i, float (*v)[8]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = i + j < i0 ? i0 : (i + j < i1 ? i + j : i1 - 1);
        if (is_v) load8<DT>(x, row(k) + 8 * c, v[j]);
        else load_rotated<DT>(a, x, row(k), c, base + k, v[j]);
      }
    };
    if (many) {
#pragma unroll 1
      for (int i = i0; i < i1; i += 4) {
        float v[4][8];
        four(i, v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[j][e]));
      }
    } else {
      for (int i = i0; i < i1; ++i) {
        float v[8];
        if (is_v) load8<DT>(x, row(i) + 8 * c, v);
        else load_rotated<DT>(a, x, row(i), c, base + i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
      }
    }
    amax = wave_max(amax);
    if constexpr (SH::kItemWaves > 1) {
      __syncthreads();
      if (lane == 0) red[wave] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < SH::kItemWaves; ++w) amax = fmaxf(amax, red[wave / SH::kItemWaves * SH::kItemWaves + w]);
    }
    if (!active || !here) continue;
    const bool fresh = lo <= lp * B;               // no token of the page is older than this call's
    const int want = exponent_byte(amax);
    const int b = fresh ? want : (had > want ? had : want);
    const int shift = fresh ? 0 : had - b;
    if (patch == 0 && b != had) *exps = (uint8_t)b;
    const int64_t at = ph * (D * B);
    uint8_t* const kc = kv.k + at + (int64_t)(kPatch * tg) * D + 8 * c;
    uint8_t* const vc = kv.v + at + (int64_t)(8 * c) * B + kPatch * tg;
    // old tokens of the patch at the new scale
    if (shift < 0 && i0 > 0) {
      if (!is_v) {
        for (int i = 0; i < i0; ++i) {
          v2i* p = (v2i*)(kc + i * D);
          const v2i o = *p;
          *p = v2i{(int)rescale4((uint32_t)o[0], shift), (int)rescale4((uint32_t)o[1], shift)};
        }
      } else {
        // 8 bytes of each feature, those past i0 kept
        for (int e = 0; e < 8; ++e) {
          v2i o = *(const v2i*)(vc + e * B);
#pragma unroll
          for (int w = 0; w < kPatch / 4; ++w) {
            const int n = i0 - 4 * w;                             // old tokens in this word
            const uint32_t mask = n >= 4 ? 0xffffffffu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
            o[w] = (int)((rescale4((uint32_t)o[w], shift) & mask) | ((uint32_t)o[w] & ~mask));
          }
          *(v2i*)(vc + e * B) = o;
        }
      }
    }
    auto codes = [&](const float* v, uint32_t& q0, uint32_t& q1) {
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = __builtin_ldexpf(v[e], 127 - b);
      q0 = pack4_e4m3(u[0], u[1], u[2], u[3]);
      q1 = pack4_e4m3(u[4], u[5], u[6], u[7]);
    };
    if (many) {
      if (!is_v) {
#pragma unroll 1
        for (int i = i0; i < i1; i += 4) {
          float v[4][8];
          four(i, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t q0, q1;
            codes(v[j], q0, q1);
            if (i + j < i1) *(v2i*)(kc + (i + j) * D) = v2i{(int)q0, (int)q1};
          }
        }
      } else {
        // the tokens of a feature together: 4 x 4 byte transpositions
        uint32_t o[8][kPatch / 4];                 // [feature][four tokens]
#pragma unroll
        for (int w = 0; w < kPatch / 4; ++w) {
          float v[4][8];
          uint32_t q[4][2];
          four(4 * w, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) codes(v[j], q[j][0], q[j][1]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t l01 = __builtin_amdgcn_perm(q[1][h], q[0][h], 0x05010400u), h01 = __builtin_amdgcn_perm(q[1][h], q[0][h], 0x07030602u);
            const uint32_t l23 = __builtin_amdgcn_perm(q[3][h], q[2][h], 0x05010400u), h23 = __builtin_amdgcn_perm(q[3][h], q[2][h], 0x07030602u);
            o[4 * h][w] = __builtin_amdgcn_perm(l23, l01, 0x05040100u);
            o[4 * h + 1][w] = __builtin_amdgcn_perm(l23, l01, 0x07060302u);
            o[4 * h + 2][w] = __builtin_amdgcn_perm(h23, h01, 0x05040100u);
            o[4 * h + 3][w] = __builtin_amdgcn_perm(h23, h01, 0x07060302u);
          }
        }
        if (i1 - i0 < kPatch) {
          // bytes of places without a new token stay (the patch is this thread's alone)
#pragma unroll
          for (int w = 0; w < kPatch / 4; ++w) {
            uint32_t put = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) put |= 4 * w + j >= i0 && 4 * w + j < i1 ? 0xffu << (8 * j) : 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e][w] = (o[e][w] & put) | (*(const uint32_t*)(vc + e * B + 4 * w) & ~put);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) *(v2i*)(vc + e * B) = v2i{(int)o[e][0], (int)o[e][1]};
      }
    } else {
      for (int i = i0; i < i1; ++i) {
        float v[8];
        uint32_t q0, q1;
        if (is_v) load8<DT>(x, row(i) + 8 * c, v);
        else load_rotated<DT>(a, x, row(i), c, base + i, v);
        codes(v, q0, q1);
        if (!is_v) {
          *(v2i*)(kc + i * D) = v2i{(int)q0, (int)q1};
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) vc[e * B + i] = (uint8_t)((e < 4 ? q0 : q1) >> (8 * (e & 3)));
        }
      }
    }
  }
}

// One new token of a sequence: D / 8 lanes hold a kv head's keys or values, 8 features each, and
// decide its scale among themselves.  `slot`: this lane's place among the sequence's heads x features.
template <int DT, int D, int B>
__device__ void append_token(const AppendArgs& a, int s, int first, int pos, int slot) {
  constexpr int kCols = D / 8;
  const KvView& kv = a.kv;
  const int item = slot / kCols, c = slot % kCols;
  const bool is_v = item >= kv.kv_heads, have = item < 2 * kv.kv_heads;
  const int head = have ? (is_v ? item - kv.kv_heads : item) : 0;
  const int lp = pos / B, off = pos % B;
  const int page = lp < kv.max_pages ? kv.table[(int64_t)s * kv.max_pages + lp] : -1;
  const bool here = page >= 0 && page < kv.num_pages;
  const int64_t ph = (int64_t)(here ? page : 0) * kv.kv_heads + head;
  uint8_t* const exps = (is_v ? kv.ve : kv.ke) + ph;
  const int had = *exps;
  float v[8];
  if (is_v) load8<DT>(a.v, (int64_t)first * a.v_stride + (int64_t)head * D + 8 * c, v);
  else load_rotated<DT>(a, a.k, (int64_t)first * a.k_stride + (int64_t)head * D, c, pos, v);
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
  // over the head's 8, 16 or 32 lanes (bit patterns of non-negative floats order as integers)
  int am = __float_as_int(amax);
  auto up = [](int x, int y) { return x > y ? x : y; };
  am = up(am, __builtin_amdgcn_update_dpp(0, am, 0xB1, 0xF, 0xF, false));
  am = up(am, __builtin_amdgcn_update_dpp(0, am, 0x4E, 0xF, 0xF, false));
  am = up(am, __builtin_amdgcn_update_dpp(0, am, 0x141, 0xF, 0xF, false));
  if constexpr (kCols >= 16) am = up(am, __builtin_amdgcn_update_dpp(0, am, 0x140, 0xF, 0xF, false));
  if constexpr (kCols >= 32) am = up(am, __shfl_xor(am, 16));
  if (!have || !here) return;
  const bool fresh = off == 0;
  const int want = exponent_byte(__int_as_float(am));
  const int b = fresh ? want : (had > want ? had : want);
  const int shift = fresh ? 0 : had - b;
  if (c == 0 && b != had) *exps = (uint8_t)b;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __builtin_ldexpf(v[e], 127 - b);
  const uint32_t q0 = pack4_e4m3(v[0], v[1], v[2], v[3]), q1 = pack4_e4m3(v[4], v[5], v[6], v[7]);
  const int64_t at = ph * (D * B);
  if (!is_v) {
    uint8_t* const codes = kv.k + at + 8 * c;
    if (shift < 0)
#pragma unroll 8
      for (int i = 0; i < off; ++i) {
        v2i* p = (v2i*)(codes + i * D);
        const v2i o = *p;
        *p = v2i{(int)rescale4((uint32_t)o[0], shift), (int)rescale4((uint32_t)o[1], shift)};
      }
    *(v2i*)(codes + off * D) = v2i{(int)q0, (int)q1};
  } else {
    uint8_t* const codes = kv.v + at + (int64_t)(8 * c) * B;
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
}

// The queries of one sequence: one token, 8 features (with pairs (i, i + r): both groups of 8 of a
// pair) and `span` heads per thread, which share their cosines and sines.
template <int DT, int D>
__device__ void rotate_queries(const AppendArgs& a, int s, int block, int blocks, int span, int threads) {
  const KvView& kv = a.kv;
  int end = kv.q_start[s + 1], first = kv.q_start[s];
  end = end < 0 ? 0 : (end > kv.tokens ? kv.tokens : end);
  first = first < 0 ? 0 : (first > end ? end : first);
  const int len = kv.kv_len[s], past = (len < 0 ? 0 : len) - (end - first);
  const int pairs = a.interleaved ? 0 : a.rot >> 4;          // units that are pairs of groups
  const int units = D / 8 - pairs, spans = (a.heads + span - 1) / span;
  const int per = units * spans;
  const int64_t all = (int64_t)(end - first) * per;
  for (int64_t i = (int64_t)block * threads + threadIdx.x; i < all; i += (int64_t)blocks * threads) {
    const int t = (int)(i / per), r = (int)(i - (int64_t)t * per);
    const int h0 = r / units * span, u = r % units;
    const bool pair = u < pairs;
    const int c = pair ? u : u + pairs;                      // (first) group of 8 features
    const bool turned = 8 * c < a.rot;
    const int pos = past + t < 0 ? 0 : past + t;
    Turn tu;
    if (turned) load_turn(a, c, pos, tu);
    const int64_t from = (int64_t)(first + t) * a.q_stride + 8 * c, to = (int64_t)(first + t) * a.heads * D + 8 * c;
    const int h1 = h0 + span < a.heads ? h0 + span : a.heads;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
      float v[8], w[8];
      load8<DT>(a.q, from + (int64_t)h * D, v);
      if (pair) {
        load8<DT>(a.q, from + (int64_t)h * D + 8 * pairs, w);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = v[e];
        turn8(tu, false, true, v, w);
        turn8(tu, false, false, w, x);
        store8<DT>(a.q_out, to + (int64_t)h * D + 8 * pairs, w);
      } else if (turned) {
        turn8(tu, true, true, v, w);
      }
      store8<DT>(a.q_out, to + (int64_t)h * D, v);
    }
  }
}

template <int DT, int D, int B>
__global__ __launch_bounds__((Shape<DT, D, B>::kThreads), 4) void k_kv_append(const AppendArgs a, int kv_blocks, int groups, int q_blocks,
                                                                                        int span, int token_blocks) {
  using SH = Shape<DT, D, B>;
  __shared__ float red[SH::kThreads / 64];
  // the pages' workgroups (few bytes, several round trips) spread evenly among the queries' (a stream):
  // workgroup i is number floor(i kv / all) of the pages' where that number grows behind it
  const int64_t all = gridDim.x, i = blockIdx.x;
  const int before = (int)(i * kv_blocks / all), after = (int)((i + 1) * kv_blocks / all);
  if (after > before) {
    if (token_blocks > 0) {
      // one new token a sequence is expected; a sequence with another number takes its pages here too
      const int s = before / token_blocks, part = before % token_blocks;
      int end = a.kv.q_start[s + 1], first = a.kv.q_start[s];
      end = end < 0 ? 0 : (end > a.kv.tokens ? a.kv.tokens : end);
      first = first < 0 ? 0 : (first > end ? end : first);
      const int pos = a.kv.kv_len[s] - 1;
      if (end - first == 1) {
        if (pos >= 0) append_token<DT, D, B>(a, s, first, pos, part * SH::kThreads + threadIdx.x);
      } else {
        for (int g = part; g < groups; g += token_blocks) append_pages<DT, D, B>(a, s, 0, g, red);
      }
    } else {
      const int b = before / groups;
      append_pages<DT, D, B>(a, b / a.reach, b % a.reach, before % groups, red);
    }
  } else {
    const int b = (int)i - before;
    rotate_queries<DT, D>(a, b / q_blocks, b % q_blocks, q_blocks, span, SH::kThreads);
  }
}

template <int DT, int D, int B>
hipError_t launch_shape(const AppendArgs& a, hipStream_t st) {
  using SH = Shape<DT, D, B>;
  const int units = a.q ? D / 8 - (a.interleaved ? 0 : a.rot >> 4) : 0;
  const AppendPlan p = append_plan(a.kv.seqs, a.max_q, a.kv.max_pages, B, a.kv.kv_heads, D, a.heads, units, SH::kItems, SH::kThreads);
  AppendArgs part = a;
  part.reach = (int)p.reach;
  for (int s = 0; s < a.kv.seqs; s += p.seqs) {
    part.kv.seqs = a.kv.seqs - s < p.seqs ? a.kv.seqs - s : p.seqs;
    part.kv.q_start = a.kv.q_start + s;
    part.kv.kv_len = a.kv.kv_len + s;
    part.kv.table = a.kv.table + (int64_t)s * a.kv.max_pages;
    const int64_t kv_blocks = p.kv_blocks(part.kv.seqs);
    k_kv_append<DT, D, B><<<(unsigned)(kv_blocks + p.q_blocks * part.kv.seqs), SH::kThreads, 0, st>>>(
        part, (int)kv_blocks, (int)p.groups, p.q_blocks > 0 ? (int)p.q_blocks : 1, p.span, (int)p.token_blocks);
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

hipError_t launch_kv_append(const AppendArgs& a, int dt, int dim, hipStream_t st) {
  switch (dt) {
    case DT_F32: return launch_dt<DT_F32>(a, dim, st);
    case DT_F16: return launch_dt<DT_F16>(a, dim, st);
    default: return launch_dt<DT_BF16>(a, dim, st);
  }
}

}  // namespace q8
