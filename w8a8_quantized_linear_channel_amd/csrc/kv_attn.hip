// Attention of new queries over the paged 8-bit key/value cache.
//
// One workgroup takes 16 RT rows (query tokens x the query heads that share a
// kv head) of one sequence and kv head and one share of the keys; its 4 waves
// take 128-key tiles in turn and join at the end.  Each wave computes
// S^T = K Q^T with v_mfma_f32_16x16x32 (16 keys x 16 rows), so lane (q, g)
// (q = lane % 16, g = lane / 16) holds scores of row q.  The keys of the eight
// 16-key MFMA tiles are dealt so that lane group g ends up with the 32
// consecutive keys 32 g .. 32 g + 31: tile t's row 4 g + i is key 32 g + 4 t + i.
// These are already the B operand of O^T = V^T P^T (contraction over keys), so
// P needs no exchange between lanes, and lane (d, g) of the A operand is 32
// consecutive bytes of a row of the value cache, whose tokens are innermost.
// K and V go from memory to registers to MFMA without LDS.
//
// e4m3 codes convert to bf16 / f16 exactly (4 significant bits).  The key
// exponent of a page multiplies the scores (one factor per lane and tile: 32
// keys lie in one page).  Values enter the product relative to the largest
// exponent byte seen so far (f16 holds 2^-24 .. 65504), which the accumulator
// is rescaled to; the softmax weights are rounded to f16 (2^-12 of a weight),
// and maximum, sum and accumulator are held in 32 bits.
#include "q8_device.hpp"
#include "q8_kv.hpp"

namespace q8 {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kTile = 128;     // keys of one wave step
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;

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

// 2^(b - 127) as a float for an exponent byte b in [0, 254]
__device__ __forceinline__ float exp_byte(int b) { return __uint_as_float(b > 0 ? (uint32_t)b << 23 : 0x400000u); }

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

template <int D, int RT, int DT>
__global__ __launch_bounds__(kThreads) void k_attn_rows(const AttnArgs a, int row_tiles, int chunk) {
  constexpr int KS = D / 32;        // MFMA steps over the features
  constexpr int NT = D / 16;        // 16-feature tiles of the output
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

  __shared__ __attribute__((aligned(16))) float s_acc[kWaves][16][D + 4];
  __shared__ float s_ml[kWaves][16][2];

  for (int r0 = tile0 * 16 * RT; r0 < rows; r0 += row_tiles * 16 * RT) {
    // the rows of this lane, one in each row tile, and the keys that they see: [low, high)
    int low[RT], high[RT];
    v4i qf[RT][KS];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = r0 + 16 * t + lr;
      const int rc = row < rows ? row : rows - 1;
      const int tok = rc / group, hq = rc - tok * group;
      const int pos = sp.past + tok;
      high[t] = a.causal ? (pos + 1 < sp.total ? pos + 1 : sp.total) : sp.total;
      low[t] = a.window > 0 ? pos - a.window + 1 : 0;
      if (row >= rows) high[t] = 0;
      const uint16_t* q = (const uint16_t*)a.q + (int64_t)(sp.first + tok) * a.q_stride +
                          (int64_t)(head * group + hq) * D + lg * (D / 4);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) qf[t][ks] = *(const v4i*)(q + 8 * ks);
    }
    // keys that any row of the tile sees
    const int last = (r0 + 16 * RT < rows ? r0 + 16 * RT : rows) - 1;
    const int pos0 = sp.past + r0 / group, pos1 = sp.past + last / group;
    int klo = a.window > 0 && pos0 - a.window + 1 > 0 ? pos0 - a.window + 1 : 0;
    int khi = a.causal ? (pos1 + 1 < sp.total ? pos1 + 1 : sp.total) : sp.total;
    // this workgroup's share: `chunk` keys from a multiple of kTile on, the last share all that is left
    const int kb0 = (klo & ~(kTile - 1)) + (split * (int64_t)chunk < khi ? split * chunk : khi);
    const int kb1 = split + 1 < (int)gridDim.x && kb0 + (int64_t)chunk < khi ? kb0 + chunk : khi;

    v4f acc[RT][NT];
    float m[RT], l[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      m[t] = -INFINITY;
      l[t] = 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[t][n] = v4f{0, 0, 0, 0};
    }
    int bmax = 0;          // the values' reference exponent byte

    for (int kb = kb0 + wave * kTile; kb < kb1; kb += kWaves * kTile) {
      // pages of the lane's K rows (chunk lr / 4) and of its own 32 keys (chunk lg);
      // a chunk without a visible key reads page 0 and is masked
      auto page_of = [&](int key) {
        const int ok = key < khi && key + 32 > klo;
        int p = ok ? kv.table[(int64_t)s * kv.max_pages + key / kv.page] : 0;
        return p < 0 ? 0 : (p >= kv.num_pages ? kv.num_pages - 1 : p);
      };
      const int keyk = kb + 32 * (lr >> 2), keyv = kb + 32 * lg;
      const int64_t ph_k = (int64_t)page_of(keyk) * kv.kv_heads + head;
      const int64_t ph_v = (int64_t)page_of(keyv) * kv.kv_heads + head;
      const uint8_t* kp = kv.k + (ph_k * kv.page + (keyk & (kv.page - 1)) + (lr & 3)) * D + lg * (D / 4);
      const uint8_t* vp = kv.v + (ph_v * D + lr) * kv.page + (keyv & (kv.page - 1));
      const float kscale = exp_byte(kv.ke[ph_v]) * a.scale_log2;
      int vb = kv.ve[ph_v];
      const bool seen = keyv < khi && keyv + 32 > klo;

      v4f sc[RT][8];
#pragma unroll
      for (int t8 = 0; t8 < 8; ++t8) {
        int kc[D / 16];
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const v4i x = *(const v4i*)(kp + (int64_t)t8 * 4 * D + 16 * i);
          kc[4 * i] = x[0]; kc[4 * i + 1] = x[1]; kc[4 * i + 2] = x[2]; kc[4 * i + 3] = x[3];
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) sc[t][t8] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const v4i kf = widen8<DT>(kc[2 * ks], kc[2 * ks + 1], 1.0f);
#pragma unroll
          for (int t = 0; t < RT; ++t) sc[t][t8] = mma16<DT>(kf, qf[t][ks], sc[t][t8]);
        }
      }
      // the values' reference exponent
      int bt = seen ? vb : 0;
      bt = max(bt, __shfl_xor(bt, 16));
      bt = max(bt, __shfl_xor(bt, 32));
      const int bnew = bt > bmax ? bt : bmax;
      const float vfix = __builtin_ldexpf(1.0f, bmax - bnew < -126 ? -126 : bmax - bnew);
      bmax = bnew;
      int down = seen ? vb - bmax : 0;
      down = down < -126 ? -126 : down;
      const float vscale = __builtin_ldexpf(1.0f, down);

      v4i pf[RT][4];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        float mx = -INFINITY;
#pragma unroll
        for (int t8 = 0; t8 < 8; ++t8)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = keyv + 4 * t8 + i;
            const float x = (key >= low[t] && key < high[t]) ? sc[t][t8][i] * kscale : -INFINITY;
            sc[t][t8][i] = x;
            mx = fmaxf(mx, x);
          }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float mn = fmaxf(m[t], mx);
        const float ref = mn == -INFINITY ? 0.0f : mn;
        const float alpha = __builtin_amdgcn_exp2f(m[t] - ref);
        m[t] = mn;
        float sum = 0.0f;
#pragma unroll
        for (int t8 = 0; t8 < 8; ++t8)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = __builtin_amdgcn_exp2f(sc[t][t8][i] - ref);
            sc[t][t8][i] = p;
            sum += p;
          }
        l[t] = l[t] * alpha + sum;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          pf[t][j] = v4i{(int)pack2_out<DT_F16>(sc[t][2 * j][0], sc[t][2 * j][1]),
                         (int)pack2_out<DT_F16>(sc[t][2 * j][2], sc[t][2 * j][3]),
                         (int)pack2_out<DT_F16>(sc[t][2 * j + 1][0], sc[t][2 * j + 1][1]),
                         (int)pack2_out<DT_F16>(sc[t][2 * j + 1][2], sc[t][2 * j + 1][3])};
        const float fix = alpha * vfix;
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[t][n] *= fix;
      }
      // bytes of keys that no row sees are cleared: they may be anything, NaN codes included
      const bool edge = kb < klo || kb + kTile > khi;
      uint32_t keep[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        uint32_t k = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = keyv + 4 * w + i;
          k |= (key >= klo && key < khi) ? 0xffu << (8 * i) : 0u;
        }
        keep[w] = edge ? k : 0xffffffffu;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const v4i x = *(const v4i*)(vp + (int64_t)(16 * n) * kv.page);
        const v4i y = *(const v4i*)(vp + (int64_t)(16 * n) * kv.page + 16);
        const int vc[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const v4i vf = widen8<DT_F16>(vc[2 * j] & (int)keep[2 * j], vc[2 * j + 1] & (int)keep[2 * j + 1], vscale);
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[t][n] = mma16<DT_F16>(vf, pf[t][j], acc[t][n]);
        }
      }
    }

    // join the four waves, one row tile at a time
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float lsum = l[t] + __shfl_xor(l[t], 16);
      lsum += __shfl_xor(lsum, 32);
      const float vtrue = exp_byte(bmax);
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n) *(v4f*)&s_acc[wave][lr][16 * n + 4 * lg] = acc[t][n] * vtrue;
      if (lg == 0) {
        s_ml[wave][lr][0] = m[t];
        s_ml[wave][lr][1] = lsum;
      }
      __syncthreads();
      // 16 threads per row, each D / 16 consecutive features
      const int row16 = tid >> 4, part = tid & 15;
      const int row = r0 + 16 * t + row16;
      if (row < rows) {
        float mm = s_ml[0][row16][0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, s_ml[w][row16][0]);
        const float ref = mm == -INFINITY ? 0.0f : mm;
        float f[kWaves], ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          f[w] = __builtin_amdgcn_exp2f(s_ml[w][row16][0] - ref);
          ll += f[w] * s_ml[w][row16][1];
        }
        const int tok = row / group, hq = row - tok * group;
        const int64_t orow = (int64_t)(sp.first + tok) * a.heads + head * group + hq;
        const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
#pragma unroll
        for (int e = 0; e < D / 16; e += 4) {
          const int d = part * 4 + (e / 4) * 64;
          v4f o = {0, 0, 0, 0};
#pragma unroll
          for (int w = 0; w < kWaves; ++w) o += *(const v4f*)&s_acc[w][row16][d] * f[w];
          if (split_out) {
            *(v4f*)(a.part + ((int64_t)split * kv.tokens * a.heads + orow) * D + d) = o;
          } else {
            o *= inv;
            *(v2i*)((uint16_t*)a.out + orow * D + d) = v2i{(int)pack2_out<DT>(o[0], o[1]), (int)pack2_out<DT>(o[2], o[3])};
          }
        }
        if (part == 0) {
          if (split_out) {
            float* ml = a.part_ml + ((int64_t)split * kv.tokens * a.heads + orow) * 2;
            ml[0] = mm;
            ml[1] = ll;
          } else if (a.lse) {
            a.lse[orow] = ll > 0.0f ? (mm + __builtin_amdgcn_logf(ll)) * 0.6931471805599453f : -INFINITY;
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- many rows
// A workgroup takes 128 rows of one sequence and kv head, 32 a wave, and goes
// through the keys in steps of 64 that it brings into LDS as codes (DMA, three
// steps ahead).  v_mfma_f32_32x32x16: S^T = K Q^T in two 32-key tiles, lane
// (q, h) (q = lane % 32, h = lane / 32) holding row q; tile T's row 8 a + 4 h + b
// is key 32 h + 16 T + 4 a + b, so that register i of tile T is key 32 h + 16 T
// + i and the weights are the B operand of O^T = V^T P^T as they stand.  Each
// wave widens the codes it reads; two workgroups share a CU, so one wave's
// softmax runs beside another's MFMAs.
//
// The running maximum is a reference that is only moved when a score passes it
// by 2^8 (weights up to 256 fit f16 and cost no precision): most steps neither
// rescale nor exchange anything between lanes.
typedef float v16 __attribute__((ext_vector_type(16)));
constexpr int kStep = 64;        // keys of one step
constexpr int kStages = 4;       // steps in LDS
constexpr int kBlockRows = 128;
constexpr int kMeta = kThreads;  // 32-key halves whose page and exponents are held at a time

template <int DT>
__device__ __forceinline__ v16 mma32(const v4i a, const v4i b, const v16 c) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// 16-byte chunk c of a key's D bytes sits at chunk c ^ key_swz: the 16 lanes that a ds_read_b128
// serves in one cycle (0-3, 12-15, 20-23, 24-27 and their complements) read 16 keys of one chunk.
template <int D>
__device__ __forceinline__ int key_swz(int key) { return D == 64 ? (key >> 2) & 3 : D == 128 ? (key >> 1) & 7 : key & 15; }
// the same of a feature's 64 value bytes
__device__ __forceinline__ int val_swz(int d) { return (d >> 2) & 3; }

template <int D, int DT>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void k_attn_tiles(const AttnArgs a, int row_tiles, int splits,
                                                                          int chunk) {
  constexpr int KS = D / 16;                     // MFMA steps over the features
  constexpr int NT = D / 32;                     // 32-feature tiles of the output
  constexpr int kTileBytes = kStep * D;          // of keys, and of values
  constexpr int kLoads = kTileBytes / 1024 / kWaves;   // DMAs of a wave for each
  __shared__ __attribute__((aligned(16))) uint8_t smem[kStages * 2 * kTileBytes];
  // page times heads plus head, and the exponent bytes (keys | values << 8), of each 32-key half of
  // up to kMeta / 2 steps: read once, so that the loop's only global loads are its DMAs
  __shared__ int s_page[kMeta], s_exp[kMeta];
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
  const int tiles = (rows + kBlockRows - 1) / kBlockRows;

  for (int tile = tiles - 1 - tile0; tile >= 0; tile -= row_tiles) {
    const int r0 = tile * kBlockRows;
    // this lane's row (rows past the end repeat the last one and are not stored)
    const int row = r0 + 32 * wave + lr, rc = row < rows ? row : rows - 1;
    const int tok = rc / group, hq = rc - tok * group;
    const int pos = sp.past + tok;
    const int high = a.causal ? (pos + 1 < sp.total ? pos + 1 : sp.total) : sp.total;
    const int low = a.window > 0 ? pos - a.window + 1 : 0;
    v4i qf[KS];
    {
      const uint16_t* q = (const uint16_t*)a.q + (int64_t)(sp.first + tok) * a.q_stride +
                          (int64_t)(head * group + hq) * D + lh * (D / 2);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[ks] = *(const v4i*)(q + 8 * ks);
        if (a.scale_log2 < 0.0f) qf[ks] ^= (int)0x80008000u;      // the sign of the scale goes into q
      }
    }
    const float scale = fabsf(a.scale_log2);
    // keys that any row of the block sees, and the range in which every row of the wave sees every key
    const int last = (r0 + kBlockRows < rows ? r0 + kBlockRows : rows) - 1;
    const int p0 = sp.past + r0 / group, p1 = sp.past + last / group;
    const int klo = a.window > 0 && p0 - a.window + 1 > 0 ? p0 - a.window + 1 : 0;
    const int khi = a.causal ? (p1 + 1 < sp.total ? p1 + 1 : sp.total) : sp.total;
    const int w0 = r0 + 32 * wave < rows ? r0 + 32 * wave : rows - 1;
    const int w1 = w0 + 31 < rows ? w0 + 31 : rows - 1;
    const int pw0 = sp.past + w0 / group, pw1 = sp.past + w1 / group;
    const int all_hi = __builtin_amdgcn_readfirstlane(a.causal ? (pw0 + 1 < sp.total ? pw0 + 1 : sp.total) : sp.total);
    const int all_lo = __builtin_amdgcn_readfirstlane(a.window > 0 ? pw1 - a.window + 1 : 0);
    const int base = klo & ~(kStep - 1);
    const int64_t from = (int64_t)split * chunk;
    const int kb0 = base + from < khi ? base + (int)from : khi;
    const int kb1 = split + 1 < splits && kb0 + (int64_t)chunk < khi ? kb0 + chunk : khi;
    const int steps = (kb1 - kb0 + kStep - 1) / kStep;

    // the lane's place in the DMAs: instruction j (0 .. 4 kLoads - 1) of a tile fills 1 KB
    uint32_t koff[kLoads], voff[kLoads];
#pragma unroll
    for (int d = 0; d < kLoads; ++d) {
      const int slot = (d * kWaves + wave) * 64 + lane;
      const int key = slot / (D / 16), f = slot / 4;
      koff[d] = (uint32_t)((key & 31) * D + (((slot % (D / 16)) ^ key_swz<D>(key)) << 4));
      voff[d] = (uint32_t)(f * kv.page) + ((uint32_t)(slot & 1) << 4 ^ (uint32_t)(val_swz(f) & 1) << 4);
    }
    // which 32-key half of the step the lane's value chunk belongs to (the same for every d)
    const bool vhalf = (((lane & 3) ^ val_swz(lane >> 2)) >> 1) != 0;
    // step i of the run of `n` that s_page describes; past its end the last one again
    auto dma = [&](int i, int n, int kb_run) {
      uint8_t* const st = smem + (i % kStages) * 2 * kTileBytes;
      i = i < n ? i : n - 1;
      const int kb = kb_run + i * kStep;
      const int ph0 = __builtin_amdgcn_readfirstlane(s_page[2 * i]), ph1 = __builtin_amdgcn_readfirstlane(s_page[2 * i + 1]);
      const int64_t o0 = kb & (kv.page - 1), o1 = (kb + 32) & (kv.page - 1);
#pragma unroll
      for (int d = 0; d < kLoads; ++d) {
        const bool second = (d * kWaves + wave) * (1024 / D) >= 32;
        const uint8_t* p = kv.k + ((int64_t)(second ? ph1 : ph0) * kv.page + (second ? o1 : o0)) * D;
        dma16(p, koff[d], st + (d * kWaves + wave) * 1024);
      }
      const uint8_t* const b0 = kv.v + (int64_t)ph0 * D * kv.page + o0;
      const uint8_t* const b1 = kv.v + (int64_t)ph1 * D * kv.page + o1;
      const uint8_t* const bv = vhalf ? b1 : b0;
#pragma unroll
      for (int d = 0; d < kLoads; ++d) dma16_ptr(bv + voff[d], st + kTileBytes + (d * kWaves + wave) * 1024);
    };

    v16 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = v16{};
    float m = -INFINITY, l = 0.0f;
    int bmax = 0;

    // operand row of key tile T: LDS key 32 h' + 16 T + 4 a + b of row 8 a + 4 h' + b
    const int key0 = 32 * ((lr >> 2) & 1) + 4 * (lr >> 3) + (lr & 3);
    const int kswz = key_swz<D>(key0);             // the same for both tiles
    auto step = [&](int i, int kb) {
      const uint8_t* const st = smem + (i % kStages) * 2 * kTileBytes;
      const int ex0 = __builtin_amdgcn_readfirstlane(s_exp[2 * i]), ex1 = __builtin_amdgcn_readfirstlane(s_exp[2 * i + 1]);
      const int v0 = ex0 >> 8, v1 = ex1 >> 8;
      // not 0: a masked score of -inf stays one
      const float kscale = fmaxf(exp_byte((lh ? ex1 : ex0) & 255) * scale, 1.17549435e-38f);
      v16 sc[2];
      v4i kx[2][D / 32];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          kx[t][c] = *(const v4i*)(st + (key0 + 16 * t) * D + (((lh * (D / 32) + c) ^ kswz) << 4));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        sc[t] = v16{};
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          sc[t] = mma32<DT>(widen8<DT>(kx[t][c][0], kx[t][c][1], 1.0f), qf[2 * c], sc[t]);
          sc[t] = mma32<DT>(widen8<DT>(kx[t][c][2], kx[t][c][3], 1.0f), qf[2 * c + 1], sc[t]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      const int keyv = kb + 32 * lh;
      if (!(kb >= all_lo && kb + kStep <= all_hi)) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int key = keyv + 16 * t + r;
            sc[t][r] = key >= low && key < high ? sc[t][r] : -INFINITY;
          }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, sc[t][r]);
      mx *= kscale;
      const int bt = v0 > v1 ? v0 : v1;
      if (__any(mx > m + 8.0f) || bt > bmax) {
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float mn = fmaxf(m, mx);
        const int bn = bt > bmax ? bt : bmax;
        int down = bmax - bn;
        down = down < -126 ? -126 : down;
        const float alpha = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.0f : mn));
        m = mn;
        bmax = bn;
        l *= alpha;
        const float fix = alpha * __builtin_ldexpf(1.0f, down);
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n] *= fix;
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      v4i pf[4];
      float sum = 0.0f;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          sc[t][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][r], kscale, -ref));
          sum += sc[t][r];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
          pf[2 * t + j] = v4i{(int)pack2_out<DT_F16>(sc[t][8 * j], sc[t][8 * j + 1]),
                              (int)pack2_out<DT_F16>(sc[t][8 * j + 2], sc[t][8 * j + 3]),
                              (int)pack2_out<DT_F16>(sc[t][8 * j + 4], sc[t][8 * j + 5]),
                              (int)pack2_out<DT_F16>(sc[t][8 * j + 6], sc[t][8 * j + 7])};
      }
      l += sum;
      int down = (lh ? v1 : v0) - bmax;
      down = down < -126 ? -126 : down;
      const float vscale = __builtin_ldexpf(1.0f, down);
      __builtin_amdgcn_sched_barrier(0);
      const uint8_t* const vr = st + kTileBytes + lr * 64;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        v4i x[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) x[t] = *(const v4i*)(vr + n * 2048 + (((2 * lh + t) ^ val_swz(lr)) << 4));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          acc[n] = mma32<DT_F16>(widen8<DT_F16>(x[t][0], x[t][1], vscale), pf[2 * t], acc[n]);
          acc[n] = mma32<DT_F16>(widen8<DT_F16>(x[t][2], x[t][3], vscale), pf[2 * t + 1], acc[n]);
        }
      }
    };
    // Value codes of keys that no row sees are cleared in LDS (they may be anything, NaN codes
    // included; their scores are masked).  Uniform over the workgroup.
    auto clear = [&](int i, int kb) {
      uint8_t* const st = smem + (i % kStages) * 2 * kTileBytes + kTileBytes;
      for (int slot = tid; slot < D * 4; slot += kThreads) {
        const int f = slot >> 2, key = kb + 16 * ((slot & 3) ^ val_swz(f));
        v4i x = *(const v4i*)(st + slot * 16);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t keep = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) keep |= key + 4 * w + e >= klo && key + 4 * w + e < khi ? 0xffu << (8 * e) : 0u;
          x[w] &= (int)keep;
        }
        *(v4i*)(st + slot * 16) = x;
      }
      __syncthreads();
    };

    for (int run = 0; run < steps; run += kMeta / 2) {
      const int n = steps - run < kMeta / 2 ? steps - run : kMeta / 2;
      const int kb_run = kb0 + run * kStep;
      {
        // a half that no row sees reads page 0 and counts as values of exponent 0
        const int key = kb_run + 32 * tid;
        const bool seen = key < khi && key + 32 > klo;
        int p = seen ? kv.table[(int64_t)s * kv.max_pages + key / kv.page] : 0;
        p = p < 0 ? 0 : (p >= kv.num_pages ? kv.num_pages - 1 : p);
        p = p * kv.kv_heads + head;
        s_page[tid] = p;
        s_exp[tid] = kv.ke[p] | (seen ? kv.ve[p] << 8 : 0);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) dma(i, n, kb_run);
      for (int i = 0; i < n; ++i) {
        // step i is this wave's oldest stage in LDS; two later ones may be on their way (past the last
        // step the DMA repeats it, so that the count is always the same)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kStages - 2) * 2 * kLoads) : "memory");
        __builtin_amdgcn_s_barrier();              // and every wave is past step i - 1
        asm volatile("" ::: "memory");
        dma(i + kStages - 1, n, kb_run);
        const int kb = kb_run + i * kStep;
        if (kb < klo || kb + kStep > khi) clear(i, kb);
        step(i, kb);
        __builtin_amdgcn_s_waitcnt(kLgkmcnt0);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
    }

    l += __shfl_xor(l, 32);
    if (row < rows) {
      const float vtrue = exp_byte(bmax);
      const int64_t orow = (int64_t)(sp.first + tok) * a.heads + head * group + hq;
      const float inv = (splits > 1 ? 1.0f : (l > 0.0f ? 1.0f / l : 0.0f)) * vtrue;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const int d = 32 * n + 2 * r + 4 * lh;
          const v4f o = {acc[n][r] * inv, acc[n][r + 1] * inv, acc[n][r + 2] * inv, acc[n][r + 3] * inv};
          if (splits > 1) *(v4f*)(a.part + ((int64_t)split * kv.tokens * a.heads + orow) * D + d) = o;
          else *(v2i*)((uint16_t*)a.out + orow * D + d) = v2i{(int)pack2_out<DT>(o[0], o[1]), (int)pack2_out<DT>(o[2], o[3])};
        }
      if (lh == 0) {
        if (splits > 1) {
          float* ml = a.part_ml + ((int64_t)split * kv.tokens * a.heads + orow) * 2;
          ml[0] = m;
          ml[1] = l;
        } else if (a.lse) {
          a.lse[orow] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f : -INFINITY;
        }
      }
    }
  }
}

// Joins the splits of a row, in their order: one wave per row of a sequence.
template <int D, int DT>
__global__ __launch_bounds__(256) void k_attn_join(const AttnArgs a, int blocks, int splits) {
  const Span sp = span_of(a, blockIdx.x / blocks);
  const int lane = threadIdx.x & 63;
  const int64_t rows = (int64_t)a.kv.tokens * a.heads, mine = (int64_t)sp.n * a.heads;
  for (int64_t r = (int64_t)(blockIdx.x % blocks) * 4 + (threadIdx.x >> 6); r < mine; r += (int64_t)blocks * 4) {
    const int64_t row = (int64_t)sp.first * a.heads + r;
    float mm = -INFINITY;
    for (int i = lane; i < splits; i += 64) mm = fmaxf(mm, a.part_ml[(i * rows + row) * 2]);
    mm = wave_max(mm);
    const float ref = mm == -INFINITY ? 0.0f : mm;
    constexpr int E = D / 64;
    float o[E] = {};
    float ll = 0.0f;
    for (int i = 0; i < splits; ++i) {
      const float* ml = a.part_ml + (i * rows + row) * 2;
      const float f = __builtin_amdgcn_exp2f(ml[0] - ref);
      ll += f * ml[1];
      const float* p = a.part + (i * rows + row) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += f * p[e];
    }
    const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) store_out<DT>(a.out, row * D + lane * E + e, o[e] * inv);
    if (a.lse && lane == 0)
      a.lse[row] = ll > 0.0f ? (mm + __builtin_amdgcn_logf(ll)) * 0.6931471805599453f : -INFINITY;
  }
}

constexpr int kSmallRows = 16;      // up to here one 16-row tile, above 128-row blocks

// How a call is cut: rows of one workgroup, row blocks of a sequence, splits of the keys and keys of
// one split.
struct Plan {
  int64_t per, blocks;
  int splits, chunk;
};
Plan plan_of(int64_t rows, int kv_heads, int seqs, int64_t max_q, int64_t max_kv, int window) {
  Plan p;
  p.per = rows > kSmallRows ? kBlockRows : kSmallRows;
  p.blocks = (rows + p.per - 1) / p.per;
  int64_t keys = max_kv;
  if (window > 0 && window + max_q + kTile < keys) keys = window + max_q + kTile;
  const int64_t groups = (int64_t)seqs * kv_heads * p.blocks;
  const int64_t step = kWaves * kTile;
  int64_t want = (1024 + groups - 1) / groups;
  const int64_t most = (keys + step - 1) / step;
  want = want > most ? most : want;
  want = want < 1 ? 1 : want;
  int64_t c = ((keys + want - 1) / want + step - 1) / step * step;
  c = c < step ? step : c;
  p.splits = (int)((keys + c - 1) / c);
  if (p.splits < 1) p.splits = 1;
  p.chunk = (int)c;
  const int64_t most_blocks = ((int64_t)1 << 30) / ((int64_t)seqs * kv_heads * p.splits);
  if (p.per == kSmallRows && p.blocks > 65535 / seqs) p.blocks = 65535 / seqs;
  if (p.blocks > most_blocks) p.blocks = most_blocks;
  if (p.blocks < 1) p.blocks = 1;
  return p;
}

template <int D, int DT>
hipError_t launch_dim(const AttnArgs& a, hipStream_t st) {
  const int64_t rows = (int64_t)a.max_q * (a.heads / a.kv.kv_heads);
  const Plan p = plan_of(rows, a.kv.kv_heads, a.kv.seqs, a.max_q, a.max_kv, a.window);
  if (p.per == kSmallRows) {
    const dim3 grid((unsigned)p.splits, (unsigned)a.kv.kv_heads, (unsigned)(p.blocks * a.kv.seqs));
    k_attn_rows<D, 1, DT><<<grid, kThreads, 0, st>>>(a, (int)p.blocks, p.chunk);
  } else {
    const unsigned grid = (unsigned)(p.blocks * a.kv.seqs * a.kv.kv_heads * p.splits);
    k_attn_tiles<D, DT><<<grid, kThreads, 0, st>>>(a, (int)p.blocks, p.splits, p.chunk);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  int64_t blocks = ((int64_t)a.max_q * a.heads + 3) / 4;
  const int64_t limit = ((int64_t)1 << 30) / a.kv.seqs;
  blocks = blocks > limit ? limit : blocks;
  k_attn_join<D, DT><<<(unsigned)(blocks * a.kv.seqs), 256, 0, st>>>(a, (int)blocks, p.splits);
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

int attn_splits(int64_t tokens, int heads, int kv_heads, int seqs, int64_t max_q, int64_t max_kv, int window) {
  (void)tokens;
  return plan_of(max_q * (heads / kv_heads), kv_heads, seqs, max_q, max_kv, window).splits;
}

hipError_t launch_attention(const AttnArgs& a, int dt, int dim, hipStream_t st) {
  return dt == DT_F16 ? launch_dt<DT_F16>(a, dim, st) : launch_dt<DT_BF16>(a, dim, st);
}

}  // namespace q8
