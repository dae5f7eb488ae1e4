// Append to the paged 8-bit key/value cache: rotate the new keys by their
// position, find each touched (page, head)'s power-of-two scale, store e4m3
// codes, and rotate the queries of the same tokens.
//
// Work is cut by page: one (sequence, touched page, kv head, K or V) is one
// item, so the scale of a page and head is decided in one place, without
// atomics, whatever the number of new tokens in it.  An item's tokens x
// features are patches of 16 tokens x 8 features, one per thread: a token's
// 8 features are one 16-byte load, K goes out as 8 bytes per token, and V,
// stored with the tokens innermost, as 16 bytes per feature, with no
// transposition through LDS.
#include "q8_device.hpp"
#include "q8_kv.hpp"

namespace q8 {
namespace {

constexpr int kThreads = 256;

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

// The 8 rotated features 8c .. 8c+7 of the head at element offset `off`.  Every
// product and the sum are rounded on their own (no contraction), so the codes
// do not depend on how the compiler pairs them.
template <int DT>
__device__ __forceinline__ void load_rotated(const AppendArgs& a, const void* x, int64_t off, int c, int pos, float* v) {
#pragma clang fp contract(off)
  load8<DT>(x, off + 8 * c, v);
  if (8 * c >= a.rot) return;
  const int half = a.rot >> 1;
  const int64_t row = (int64_t)(pos < a.positions ? pos : a.positions - 1) * half;
  if (a.interleaved) {
    const v4f co = *(const v4f*)(a.cos + row + 4 * c), si = *(const v4f*)(a.sin + row + 4 * c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = v[2 * i], r = v[2 * i + 1];
      v[2 * i] = p * co[i] - r * si[i];
      v[2 * i + 1] = r * co[i] + p * si[i];
    }
  } else {
    const bool low = 8 * c < half;
    const int j = low ? 8 * c : 8 * c - half;
    float w[8], co[8], si[8];
    load8<DT>(x, off + (low ? 8 * c + half : 8 * c - half), w);
    load8<DT_F32>(a.cos, row + j, co);
    load8<DT_F32>(a.sin, row + j, si);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = low ? v[i] * co[i] - w[i] * si[i] : v[i] * co[i] + w[i] * si[i];
  }
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
  static constexpr int kPatches = (B / 16) * kCols;              // of one item
  static constexpr int kItemWaves = kPatches > 64 ? kPatches / 64 : 1;
  static constexpr int kItems = kThreads / 64 / kItemWaves;      // items of one workgroup
  static_assert(kItemWaves <= kThreads / 64, "an item fits one workgroup");
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
    const int page = kv.table[(int64_t)s * kv.max_pages + lp];
    if (page < 0 || page >= kv.num_pages) continue;
    const int base = lp * B + 16 * tg;
    int i0 = lo - base, i1 = hi - base;
    i0 = i0 < 0 ? 0 : (i0 > 16 ? 16 : i0);
    i1 = i1 < 0 ? 0 : (i1 > 16 ? 16 : i1);
    const bool active = have && patch < SH::kPatches;
    if (!active) i0 = i1 = 0;
    auto row = [&](int i) { return (int64_t)(first + (base + i - past)) * stride + (int64_t)head * D; };
    float amax = 0.0f;
    for (int i = i0; i < i1; ++i) {
      float v[8];
      if (is_v) load8<DT>(x, row(i) + 8 * c, v);
      else load_rotated<DT>(a, x, row(i), c, base + i, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
    }
    amax = wave_max(amax);
    if constexpr (SH::kItemWaves > 1) {
      __syncthreads();
      if (lane == 0) red[wave] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < SH::kItemWaves; ++w) amax = fmaxf(amax, red[wave / SH::kItemWaves * SH::kItemWaves + w]);
    }
    if (!active) continue;
    uint8_t* const exps = (is_v ? kv.ve : kv.ke) + (int64_t)page * kv.kv_heads + head;
    const bool fresh = lo <= lp * B;               // no token of the page is older than this call's
    const int want = exponent_byte(amax), had = *exps;
    const int b = fresh ? want : (had > want ? had : want);
    const int shift = fresh ? 0 : had - b;
    if (patch == 0 && b != had) *exps = (uint8_t)b;
    const int64_t at = ((int64_t)page * kv.kv_heads + head) * (D * B);
    if (!is_v) {
      uint8_t* const codes = kv.k + at + (int64_t)(16 * tg) * D + 8 * c;
      if (shift < 0)
        for (int i = 0; i < i0; ++i) {
          v2i* p = (v2i*)(codes + i * D);
          const v2i o = *p;
          *p = v2i{(int)rescale4((uint32_t)o[0], shift), (int)rescale4((uint32_t)o[1], shift)};
        }
      for (int i = i0; i < i1; ++i) {
        float v[8];
        load_rotated<DT>(a, x, row(i), c, base + i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_ldexpf(v[e], 127 - b);
        *(v2i*)(codes + i * D) = v2i{(int)pack4_e4m3(v[0], v[1], v[2], v[3]), (int)pack4_e4m3(v[4], v[5], v[6], v[7])};
      }
    } else {
      uint8_t* const codes = kv.v + at + (int64_t)(8 * c) * B + 16 * tg;
      if (shift < 0 && i0 > 0) {
        // old tokens of the patch: 16 bytes of each feature, those past i0 kept
        for (int e = 0; e < 8; ++e) {
          v4i o = *(const v4i*)(codes + e * B);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int n = i0 - 4 * w;                             // old tokens in this word
            const uint32_t mask = n >= 4 ? 0xffffffffu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
            o[w] = (int)((rescale4((uint32_t)o[w], shift) & mask) | ((uint32_t)o[w] & ~mask));
          }
          *(v4i*)(codes + e * B) = o;
        }
      }
      if (i0 == 0 && i1 == 16) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t q[4][2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v[8];
            load8<DT>(x, row(4 * w + i) + 8 * c, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __builtin_ldexpf(v[e], 127 - b);
            q[i][0] = pack4_e4m3(v[0], v[1], v[2], v[3]);
            q[i][1] = pack4_e4m3(v[4], v[5], v[6], v[7]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t sel = 8 * (e & 3);
            uint32_t r = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) r |= ((q[i][e >> 2] >> sel) & 0xffu) << (8 * i);
            *(uint32_t*)(codes + e * B + 4 * w) = r;
          }
        }
      } else {
        for (int i = i0; i < i1; ++i) {
          float v[8];
          load8<DT>(x, row(i) + 8 * c, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __builtin_ldexpf(v[e], 127 - b);
          const uint32_t q0 = pack4_e4m3(v[0], v[1], v[2], v[3]), q1 = pack4_e4m3(v[4], v[5], v[6], v[7]);
#pragma unroll
          for (int e = 0; e < 8; ++e) codes[e * B + i] = (uint8_t)((e < 4 ? q0 : q1) >> (8 * (e & 3)));
        }
      }
    }
  }
}

// The queries of one sequence: one (token, head, 8 features) per thread.
template <int DT, int D>
__device__ void rotate_queries(const AppendArgs& a, int s, int block, int blocks) {
  const KvView& kv = a.kv;
  int end = kv.q_start[s + 1], first = kv.q_start[s];
  end = end < 0 ? 0 : (end > kv.tokens ? kv.tokens : end);
  first = first < 0 ? 0 : (first > end ? end : first);
  const int len = kv.kv_len[s], past = (len < 0 ? 0 : len) - (end - first);
  const int per = a.heads * (D / 8);
  const int64_t all = (int64_t)(end - first) * per;
  for (int64_t i = (int64_t)block * kThreads + threadIdx.x; i < all; i += (int64_t)blocks * kThreads) {
    const int t = (int)(i / per), r = (int)(i - (int64_t)t * per);
    const int h = r / (D / 8), c = r % (D / 8);
    const int pos = past + t < 0 ? 0 : past + t;
    float v[8];
    load_rotated<DT>(a, a.q, (int64_t)(first + t) * a.q_stride + (int64_t)h * D, c, pos, v);
    store8<DT>(a.q_out, ((int64_t)(first + t) * a.heads + h) * D + 8 * c, v);
  }
}

template <int DT, int D, int B>
__global__ __launch_bounds__(kThreads) void k_kv_append(const AppendArgs a, int kv_blocks, int groups, int q_blocks) {
  __shared__ float red[kThreads / 64];
  int b = blockIdx.x;
  if (b < kv_blocks) {
    const int group = b % groups;
    b /= groups;
    append_pages<DT, D, B>(a, b / a.reach, b % a.reach, group, red);
  } else {
    b -= kv_blocks;
    rotate_queries<DT, D>(a, b / q_blocks, b % q_blocks, q_blocks);
  }
}

template <int DT, int D, int B>
hipError_t launch_shape(const AppendArgs& a, hipStream_t st) {
  using SH = Shape<DT, D, B>;
  const int64_t groups = (2 * a.kv.kv_heads + SH::kItems - 1) / SH::kItems;
  const int64_t kv_blocks = (int64_t)a.kv.seqs * a.reach * groups;
  int64_t q_blocks = 0;
  if (a.q) {
    q_blocks = ((int64_t)a.max_q * a.heads * (D / 8) + kThreads - 1) / kThreads;
    const int64_t most = ((int64_t)1 << 30) / a.kv.seqs;
    q_blocks = q_blocks > most ? most : q_blocks;
  }
  if (kv_blocks + q_blocks * a.kv.seqs > ((int64_t)1 << 31) - 1) return hipErrorInvalidValue;
  k_kv_append<DT, D, B><<<(unsigned)(kv_blocks + q_blocks * a.kv.seqs), kThreads, 0, st>>>(a, (int)kv_blocks, (int)groups,
                                                                                          q_blocks > 0 ? (int)q_blocks : 1);
  return hipGetLastError();
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
