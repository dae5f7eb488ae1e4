// FP8 e4m3 product with a scale for each block of 128: activations [M, K]
// carry one scale per token and 128 features, weights [N, K] one per block of
// 128 rows x 128 features:
//     y[m,n] = sum_j S_x[j,m] S_w[n / 128, j] sum_{k in j} e4m3(xq[m,k]) e4m3(wq[n,k])  (+ b[n])
// Each block's inner sum is one chain of MFMAs started at zero, multiplied by
// its scale in fp32 and added to the fp32 accumulator.
#include <type_traits>

#include "q8_device.hpp"
#include "q8_kv.hpp"

namespace q8 {
namespace {

constexpr int kThreads = 256;

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

// max(a, |b|), a NaN if either is: a block with a NaN gets a NaN scale, so that what is computed from it
// is NaN, too (the clamp of the codes would make -448 of it)
__device__ __forceinline__ float amax_of(float a, float b) { return __builtin_elementwise_maximum(a, fabsf(b)); }
// of non-negative floats or NaN, whose bit patterns order as integers
__device__ __forceinline__ int bits_max(int a, int b) { return a > b ? a : b; }

// e4m3 codes of 8 values, x / s rounded as the correctly rounded quotient is
// (16-bit inputs: two FMAs on RN(1/s), the same codes over that whole domain)
template <int DT>
__device__ __forceinline__ v2i codes8(const float* v, float s) {
  const float r = 1.0f / s;
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = DT == DT_F32 ? v[e] / s : __builtin_copysignf(quot_fma(v[e], s, r), v[e]);
    q[e] = fminf(fmaxf(y, -kFp8Max), kFp8Max);
  }
  return v2i{(int)pack4_e4m3(q[0], q[1], q[2], q[3]), (int)pack4_e4m3(q[4], q[5], q[6], q[7])};
}

// One 16-lane row of a wave per group of 128 features of one token.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_quant_act_block(const void* __restrict__ x, int64_t M, int64_t K, int groups,
                                                              uint8_t* __restrict__ xq, float* __restrict__ x_scale) {
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
  if (i >= M * groups) return;                                 // whole 16-lane rows leave together
  const int64_t m = i / groups;
  const int j = (int)(i - m * groups), k = j * kScaleBlock + 8 * (threadIdx.x & 15);
  float v[8] = {};
  if (k < K) load8<DT>(x, m * K + k, v);
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = amax_of(amax, v[e]);
  amax = __int_as_float(dpp_row_reduce(__float_as_int(fabsf(amax)), bits_max));
  float s = amax / kFp8Max;
  s = s < kEps ? kEps : s;
  if (k < K) *(v2i*)(xq + m * K + k) = codes8<DT>(v, s);
  if ((threadIdx.x & 15) == 0) x_scale[(int64_t)j * M + m] = s;
}

// One workgroup per 128 x 128 block of the weights (offline).
template <int DT>
__global__ __launch_bounds__(kThreads) void k_quant_weight_block(const void* __restrict__ w, int64_t N, int64_t K,
                                                                 uint8_t* __restrict__ wq, float* __restrict__ w_scale) {
  __shared__ int red[kThreads / 64];
  const int cols = (int)((K + kScaleBlock - 1) / kScaleBlock);
  const int64_t n0 = (int64_t)(blockIdx.x / cols) * kScaleBlock;
  const int k = (int)(blockIdx.x % cols) * kScaleBlock + 8 * (threadIdx.x & 15);
  const int r0 = threadIdx.x >> 4;
  float amax = 0.0f;
  for (int r = r0; r < kScaleBlock; r += kThreads / 16) {
    if (n0 + r >= N || k >= K) continue;
    float v[8];
    load8<DT>(w, (n0 + r) * K + k, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = amax_of(amax, v[e]);
  }
  int top = dpp_row_reduce(__float_as_int(fabsf(amax)), bits_max);
  top = bits_max(bits_max(__builtin_amdgcn_readlane(top, 0), __builtin_amdgcn_readlane(top, 16)),
                 bits_max(__builtin_amdgcn_readlane(top, 32), __builtin_amdgcn_readlane(top, 48)));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) top = bits_max(top, red[w]);
  amax = __int_as_float(top);
  float s = amax / kFp8Max;
  s = s < kEps ? kEps : s;
  for (int r = r0; r < kScaleBlock; r += kThreads / 16) {
    if (n0 + r >= N || k >= K) continue;
    float v[8];
    load8<DT>(w, (n0 + r) * K + k, v);
    *(v2i*)(wq + (n0 + r) * K + k) = codes8<DT_F32>(v, s);
  }
  if (threadIdx.x == 0) w_scale[blockIdx.x] = s;
}

// ---------------------------------------------------------------- tiles
// Y tiles of BM x BN by WM x WN waves, each AF x BF fragments of 16 x 16
// (v_mfma_f32_16x16x128_f8f6f4, weights first: a fragment holds D[n][m], lane l
// four rows n of column m = l % 16).  One instruction is one scale block, so a
// block's sums start from zero, are multiplied by S_x S_w and added to the
// accumulator with no second instruction in between (the 32 x 32 x 64 shape
// needs two, and four times the registers for the sums: 243 against 233 us at
// 4096 x 4096 x 14336 in the kernel trace).
// One stage is one block, 128 bytes of K of every tile row, filled by LDS DMA
// with the block's activation scales of the tile beside it.  The last block
// goes the same way and is cut at K in registers (a pass of its own through
// registers: 11.0 against 9.9 us at 333 x 1000 x 2064).
//
// 256 x 256 tiles, 4096 x 4096 x 14336: 210 to 250 us as the clock allows (481 G
// flop, 1.9 to 2.3 PFLOP/s), bound by the matrix units and the fp32 multiply-add
// that every 128-deep sum needs; tiles of 256 x 128 and 128 x 256 257 and 259 us
// against 222, a prefetch into L2 240.  Small
// tiles are bound by what a step costs: its barrier, DMA requests and LDS reads.
constexpr int kBK = kScaleBlock;
constexpr int kXcds = 8;
constexpr int kGroupM = 4;       // tile rows that share weight tiles in L2

// 128-byte LDS rows, the 16-byte chunk c of row r at c ^ ((r >> 1) & 7): the 16
// rows that a fragment read touches in one cycle cover all 64 banks once.
__device__ __forceinline__ int swz_key(int row) { return (row >> 1) & 7; }

// LDS DMA through a buffer resource: 64 lanes x 16 (or 4) bytes from base + voff (per lane) + soff
// into consecutive LDS; bytes past the resource's end arrive as zeros.  Inline asm for the reason
// given at dma16 (q8_device.hpp); callers wait with vmcnt.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16_buf(v4i rsrc, uint32_t voff, uint32_t soff, void* lds) {
  const uint32_t m0 = (uint32_t)(uintptr_t)(lptr_t)lds;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(m0), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}
__device__ __forceinline__ void dma4_buf(v4i rsrc, uint32_t voff, uint32_t soff, void* lds) {
  const uint32_t m0 = (uint32_t)(uintptr_t)(lptr_t)lds;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(m0), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}
#pragma clang diagnostic pop
// Words of a raw byte buffer over [p, p + bytes)
__device__ __forceinline__ v4i buffer_words(const void* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)p;
  return v4i{__builtin_amdgcn_readfirstlane((int)(uint32_t)a), __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
             __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

template <int BM, int BN, int WM, int WN, int NST>
struct Tile {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int TM = BM / WM, TN = BN / WN, AF = TM / 16, BF = TN / 16, H = AF / 2;
  static constexpr int kStage = (BM + BN) * kBK;
  static constexpr int kLoads = (BM + BN) / 8 / kWaves;    // 1 KB DMAs (8 rows) of a wave and stage
  static constexpr int kScales = BM / 64;                  // 64-row DMAs of activation scales of a stage
  static constexpr bool kAhead = AF * BF <= 8;             // a whole block ahead in registers
  static constexpr int kScaleBytes = (BM + (kAhead ? 64 : 0)) * 4;
  static constexpr int kPitch = TN * 4 + 16;               // epilogue staging of one 16-row slab
  static constexpr int kLds = NST * (kStage + kScaleBytes);
  static_assert((BM + BN) / 8 % kWaves == 0 && BM % 64 == 0 && kScales + kAhead <= kWaves, "DMA split");
  static_assert(kWaves * 16 * kPitch <= kLds, "the epilogue's staging fits");
};

template <int BM, int BN, int WM, int WN, int NST, int YDT>
__global__ __launch_bounds__(64 * WM * WN, WM * WN / 4) void k_gemm_tiles(
    const uint8_t* __restrict__ xq, const float* __restrict__ x_scale, int M, int K, const uint8_t* __restrict__ wq,
    const float* __restrict__ w_scale, int N, const float* __restrict__ bias, void* __restrict__ y) {
  using TL = Tile<BM, BN, WM, WN, NST>;
  constexpr int AF = TL::AF, BF = TL::BF, H = TL::H;
  static_assert(AF % 2 == 0 && TL::TN <= kScaleBlock, "wave tile");
  __shared__ __attribute__((aligned(16))) uint8_t smem[TL::kLds];
  float* const ssc = (float*)(smem + NST * TL::kStage);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;

  // XCD-contiguous renumbering of the tiles, kGroupM tile rows to a column group
  const int ntm = (M + BM - 1) / BM, ntn = (N + BN - 1) / BN;
  int m0, n0;
  {
    const int T = ntm * ntn, q = T / kXcds, r = T % kXcds;
    const int x = blockIdx.x % kXcds, i = blockIdx.x / kXcds;
    const int b = x * q + (x < r ? x : r) + i;
    const int per = kGroupM * ntn, g = b / per, first = g * kGroupM;
    const int size = ntm - first < kGroupM ? ntm - first : kGroupM;
    m0 = (first + (b - g * per) % size) * BM;
    n0 = (b - g * per) / size * BN;
  }
  const int groups = (K + kBK - 1) / kBK;

  // DMA: instruction d of this wave fills rows 8 (d kWaves + wave) .. + 7 of the stage (activation
  // rows first); lane l lands at row l / 8, chunk l % 8, and fetches the chunk that belongs there.
  // Rows past M or N read what follows (zeros past the arrays) and feed outputs that are not stored.
  constexpr int kStep = TL::kWaves * 8;                      // rows from one DMA to the next
  const int r0 = wave * 8 + (lane >> 3);
  const uint32_t chunk = (uint32_t)((lane & 7) ^ swz_key(r0)) << 4;
  const uint32_t offx = (uint32_t)(m0 + r0) * (uint32_t)K + chunk, offw = (uint32_t)(n0 + r0) * (uint32_t)K + chunk;
  // scales: 64 rows' of the activations, or (kAhead) the one of the tile's weight rows 64 times
  const int part = wave % (TL::kScales + TL::kAhead);
  const bool wpart = TL::kAhead && part == TL::kScales;
  const uint32_t offs = wpart ? (uint32_t)(n0 / kScaleBlock) * (uint32_t)groups * 4u : (uint32_t)(m0 + part * 64 + lane) * 4u;
  const v4i resx = buffer_words(xq, (uint32_t)M * (uint32_t)K), resw = buffer_words(wq, (uint32_t)N * (uint32_t)K);
  const v4i ress = buffer_words(wpart ? w_scale : x_scale,
                                (wpart ? (uint32_t)((N + kScaleBlock - 1) / kScaleBlock) : (uint32_t)M) * (uint32_t)groups * 4u);
  const uint32_t steps = (wpart ? 1u : (uint32_t)M) * 4u;
  // instruction d of block j's kLoads + 1
  auto dma_one = [&](int j, int slot, int d) {
    if (d == TL::kLoads) {
      dma4_buf(ress, offs, (uint32_t)j * steps, ssc + slot * (TL::kScaleBytes / 4) + part * 64);
      return;
    }
    const bool w = d * kStep >= BM;
    // the row step belongs to the per-lane offset: the range check takes the scalar one off the size
    const uint32_t step = (uint32_t)(w ? d * kStep - BM : d * kStep) * (uint32_t)K;
    dma16_buf(w ? resw : resx, (w ? offw : offx) + step, (uint32_t)j * kBK,
              smem + slot * TL::kStage + wave * 1024 + d * TL::kWaves * 1024);
  };
  auto dma = [&](int j, int slot) {
#pragma unroll
    for (int d = 0; d <= TL::kLoads; ++d) dma_one(j, slot, d);
  };
  v4f acc[AF][BF];
#pragma unroll
  for (int i = 0; i < AF; ++i)
#pragma unroll
    for (int f = 0; f < BF; ++f) acc[i][f] = v4f{0, 0, 0, 0};

  // operand of row base + lane % 16: logical chunks lane / 16 and lane / 16 + 4 (any split of the block
  // does that both operands share).  A ds_read_b128 serves lanes 0-3, 12-15, 20-23 and 24-27 in one
  // cycle: rows 0-3 and 12-15 of one chunk with rows 4-11 of the next are all 64 banks once; with
  // chunks 2 (lane / 16) and 2 (lane / 16) + 1 every read took two turns.
  const int lr = lane & 15, lg = lane >> 4;
  const int lo = lr * kBK + ((lg ^ swz_key(lr)) << 4), lo2 = lo ^ 64;
  const uint8_t* const sx_rows = smem + wm * TL::TM * kBK;
  const uint8_t* const sw_rows = smem + (BM + wn * TL::TN) * kBK;
  auto frag = [&](const uint8_t* rows) {
    const v4i a = *(const v4i*)(rows + lo), b = *(const v4i*)(rows + lo2);
    return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  };
  auto mma = [&](const v8i& w, const v8i& x) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
  };
  auto add = [&](int i, int f, float s, const v4f p) {
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[i][f][r] = __builtin_fmaf(s, p[r], acc[i][f][r]);
  };
  // K may end inside the last block, whose LDS rows then go on with what follows in memory, another
  // row's codes: they are cleared on both sides (a NaN among them stays in its own row)
  const int chunks = (K - (groups - 1) * kBK) >> 4, keep_lo = lg < chunks ? -1 : 0, keep_hi = lg + 4 < chunks ? -1 : 0;
  auto cut = [&](v8i& v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] &= keep_lo;
      v[4 + e] &= keep_hi;
    }
  };
  // All NST buffers are filled ahead, a buffer again as soon as every wave has read its block.  Past
  // the last block the DMA repeats it, into buffers nobody reads, so that the loop has no
  // branch and the number of loads in flight is always the same.
  auto arrived = [&] {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 2) * (TL::kLoads + 1)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto clamped = [&](int b) { return b < groups ? b : groups - 1; };
#pragma unroll
  for (int b = 0; b < NST - 1; ++b) dma(clamped(b), b);
  arrived();
  dma(clamped(NST - 1), NST - 1);
  if constexpr (TL::kAhead) {
    // Small wave tiles: the next block's operands go from LDS into a second set of registers and the
    // DMA of a later one is requested while this block's products run, a few requests after each
    // (all of them before the products: 70.9 against 55.9 us for 128 x 128 tiles at 512 x 2048 x
    // 16384, where nothing but this loop counts).
    v8i fa[2][AF], fb[2][BF];
    float sx[2][AF], sw[2];
    constexpr int kReads = AF + BF + 1, kProducts = AF * BF, kOps = kReads + TL::kLoads + 1;
    // read r of a block's kReads: its scales, a weight or an activation fragment
    auto read = [&](int slot, auto SET, int r) {
      constexpr int t = decltype(SET)::value;
      const float* const sc = ssc + slot * (TL::kScaleBytes / 4);
      if (r == 0) {
#pragma unroll
        for (int i = 0; i < AF; ++i) sx[t][i] = sc[wm * TL::TM + 16 * i + lr];
        sw[t] = sc[BM];
      } else if (r <= BF) {
        fb[t][r - 1] = frag(sw_rows + slot * TL::kStage + (r - 1) * 16 * kBK);
      } else {
        fa[t][r - 1 - BF] = frag(sx_rows + slot * TL::kStage + (r - 1 - BF) * 16 * kBK);
      }
    };
    // The block of SET multiplied; after product c, `between(c)`.
    auto multiply = [&](auto SET, auto&& between) {
      constexpr int t = decltype(SET)::value;
      v4f p[AF][BF];
#pragma unroll
      for (int c = 0; c < kProducts; ++c) {
        p[c / BF][c % BF] = mma(fb[t][c % BF], fa[t][c / BF]);
        __builtin_amdgcn_sched_barrier(0);
        between(c);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int c = 0; c < kProducts; ++c) add(c / BF, c % BF, sx[t][c / BF] * sw[t], p[c / BF][c % BF]);
    };
    auto last = [&](auto SET) {
      constexpr int t = decltype(SET)::value;
#pragma unroll
      for (int i = 0; i < AF; ++i) cut(fa[t][i]);
#pragma unroll
      for (int f = 0; f < BF; ++f) cut(fb[t][f]);
      multiply(SET, [](int) {});
    };
    constexpr std::integral_constant<int, 0> even;
    constexpr std::integral_constant<int, 1> odd;
    auto step = [&](int j, auto SET, auto NEXT) {
      __builtin_amdgcn_s_waitcnt(kLgkmcnt0);            // this wave's reads of block j are done
      arrived();
      const int from = (j + 1) % NST, to = j % NST, b = clamped(j + NST);
      multiply(SET, [&](int c) {
#pragma unroll
        for (int o = c * kOps / kProducts; o < (c + 1) * kOps / kProducts; ++o) {
          if (o < kReads) read(from, NEXT, o);
          else dma_one(b, to, o - kReads);
        }
      });
    };
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(0, even, r);
    int j = 0;
    for (; j + 2 < groups; j += 2) {
      step(j, even, odd);
      step(j + 1, odd, even);
    }
    if (j + 1 < groups) {
      step(j, even, odd);
      last(odd);
    } else {
      last(even);
    }
  } else {
    // the wave's columns lie in one block of 128 weight rows
    const int nw = n0 + wn * TL::TN < N ? n0 + wn * TL::TN : N - 1;
    const float* const wsc = w_scale + (int64_t)(nw / kScaleBlock) * groups;

    // The block's weight fragments and half of its activation fragments are in registers; a fragment's
    // registers are loaded again as soon as its last MFMA is issued, so LDS reads run all the time and a
    // wave leaves the barrier with the second half of a block still to multiply.
    float sw, swn, sx[H];
    v8i fb[BF], fa[H];
    auto load_b = [&](int slot, int f) { fb[f] = frag(sw_rows + slot * TL::kStage + f * 16 * kBK); };
    auto load_a = [&](int slot, int h, int i) {
      fa[h] = frag(sx_rows + slot * TL::kStage + i * 16 * kBK);
      sx[h] = ssc[slot * (TL::kScaleBytes / 4) + wm * TL::TM + 16 * i + lr];
    };
    // A block; `next` (uniform) runs once this wave has read all of it and returns the slot that the
    // registers are filled from.  The last block (not NEXT) fills none and is cut at K.
    auto block = [&](int slot, auto NEXT, auto&& next) {
      constexpr bool more = decltype(NEXT)::value;
      sw = swn;
      if (!more) {
#pragma unroll
        for (int h = 0; h < H; ++h) cut(fa[h]);
#pragma unroll
        for (int f = 0; f < BF; ++f) cut(fb[f]);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        v4f p[BF];
#pragma unroll
        for (int f = 0; f < BF; ++f) p[f] = mma(fb[f], fa[h]);
        const float s = sx[h] * sw;
        __builtin_amdgcn_sched_barrier(0);
        load_a(slot, h, H + h);
        if (!more) cut(fa[h]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < BF; ++f) add(h, f, s, p[f]);
        __builtin_amdgcn_sched_barrier(0);
      }
      const int to = next();
      float s[H];
#pragma unroll
      for (int h = 0; h < H; ++h) s[h] = sx[h] * sw;
#pragma unroll
      for (int d = 0; d < (H > BF ? H : BF); ++d) {
        v4f p[H], q[BF];
        if (d < BF) {
#pragma unroll
          for (int h = d; h < H; ++h) p[h] = mma(fb[d], fa[h]);
          __builtin_amdgcn_sched_barrier(0);
          if (more) load_b(to, d);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (d < H) {
#pragma unroll
          for (int f = d + 1; f < BF; ++f) q[f] = mma(fb[f], fa[d]);
          __builtin_amdgcn_sched_barrier(0);
          if (more) load_a(to, d, d);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (d < BF) {
#pragma unroll
          for (int h = d; h < H; ++h) add(H + h, d, s[h], p[h]);
        }
        if (d < H) {
#pragma unroll
          for (int f = d + 1; f < BF; ++f) add(H + d, f, s[d], q[f]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto load_all = [&](int slot, int j) {
#pragma unroll
      for (int f = 0; f < BF; ++f) load_b(slot, f);
#pragma unroll
      for (int h = 0; h < H; ++h) load_a(slot, h, h);
      swn = wsc[j];
    };

    load_all(0, 0);
    int j = 0;
    for (; j + 1 < groups; ++j)
      block(j % NST, std::true_type{}, [&] {
        __builtin_amdgcn_s_waitcnt(kLgkmcnt0);          // this wave's reads of block j are done
        arrived();
        dma(clamped(j + NST), j % NST);
        swn = wsc[j + 1];
        return (j + 1) % NST;
      });
    block(j % NST, std::false_type{}, [] { return 0; });
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // repeated blocks still on their way

  // epilogue: one 16-row slab of a wave at a time through padded LDS, back row-contiguous, 8 columns a lane
  __syncthreads();
  constexpr int kPitch = TL::kPitch, LPR = TL::TN / 8, RPI = 64 / LPR;
  uint8_t* const stg = smem + wave * 16 * kPitch;
  const int rc = lane % LPR, rr = lane / LPR;
  const int n = n0 + wn * TL::TN + 8 * rc;
  float b8[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) b8[e] = bias && n + e < N ? bias[n + e] : 0.0f;
  const bool vec = (N & 7) == 0;
#pragma unroll
  for (int i = 0; i < AF; ++i) {
#pragma unroll
    for (int f = 0; f < BF; ++f) *(v4f*)(stg + lr * kPitch + (16 * f + 4 * lg) * 4) = acc[i][f];
#pragma unroll
    for (int t = 0; t < (16 + RPI - 1) / RPI; ++t) {
      const int row = t * RPI + rr, m = m0 + wm * TL::TM + 16 * i + row;
      if (row >= 16 || m >= M || n >= N) continue;
      const v4f a = *(const v4f*)(stg + row * kPitch + rc * 32), b = *(const v4f*)(stg + row * kPitch + rc * 32 + 16);
      const float v[8] = {a[0] + b8[0], a[1] + b8[1], a[2] + b8[2], a[3] + b8[3],
                          b[0] + b8[4], b[1] + b8[5], b[2] + b8[6], b[3] + b8[7]};
      uint16_t* const o = (uint16_t*)y + (int64_t)m * N + n;
      if (vec) {
        const v4i p = {(int)pack2_out<YDT>(v[0], v[1]), (int)pack2_out<YDT>(v[2], v[3]), (int)pack2_out<YDT>(v[4], v[5]),
                       (int)pack2_out<YDT>(v[6], v[7])};
        __builtin_nontemporal_store(p, (v4i*)o);
      } else {
        for (int e = 0; e < 8 && n + e < N; ++e) store_out<YDT>(o, e, v[e]);
      }
    }
  }
}

// ---------------------------------------------------------------- few tokens
// Decode-shaped: a workgroup owns 16 weight rows, its 4 waves take every fourth
// block of K (v_mfma_f32_16x16x128_f8f6f4: one block an instruction), AHEAD
// blocks at a time, all of whose weights and activations are requested before
// the first is used, straight into registers, and join through LDS.  MF
// fragments of 16 tokens share a weight operand.  Bound by latency and the
// weights' bytes (16 tokens, 4096 x 4096: 6.2 us, 2.7 TB/s).
constexpr int kGemvWaves = kThreads / 64;

// Joins the waves' sums of a 16 x 16 MF tile and stores them.
template <int MF, int YDT>
__device__ __forceinline__ void gemv_store(v4f (&acc)[MF], v4f (*part)[MF][64], int wave, int lane, int M, int N, int n0,
                                           const float* bias, void* y) {
#pragma unroll
  for (int f = 0; f < MF; ++f) part[wave][f][lane] = acc[f];
  __syncthreads();
  const int lr = lane & 15, lg = lane >> 4;
  const int m = 16 * wave + lr, n4 = n0 + 4 * lg;
  if (wave >= MF || m >= M) return;
  v4f t = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < kGemvWaves; ++w) t += part[w][wave][lane];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n4 + r < N) store_out<YDT>(y, (int64_t)m * N + n4 + r, t[r] + (bias ? bias[n4 + r] : 0.0f));
}

__device__ __forceinline__ v8i join8(const v4i a, const v4i b) {
  return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

template <int MF, int AHEAD, int YDT>
__global__ __launch_bounds__(kThreads) void k_gemv_block(const uint8_t* __restrict__ xq, const float* __restrict__ x_scale,
                                                         int M, int K, const uint8_t* __restrict__ wq,
                                                         const float* __restrict__ w_scale, int N,
                                                         const float* __restrict__ bias, void* __restrict__ y) {
  static_assert(MF <= kGemvWaves, "a wave a fragment at the join");
  __shared__ v4f part[kGemvWaves][MF][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int groups = (K + kScaleBlock - 1) / kScaleBlock;
  // rows past N and tokens past M read the last ones and are not stored
  const int n = n0 + lr < N ? n0 + lr : N - 1;
  const uint8_t* const wp = wq + (int64_t)n * K + 32 * lg;
  const float* const ws = w_scale + (int64_t)(n0 / kScaleBlock) * groups;
  const uint8_t* xp[MF];
  const float* xs[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int m = 16 * f + lr < M ? 16 * f + lr : M - 1;
    xp[f] = xq + (int64_t)m * K + 32 * lg;
    xs[f] = x_scale + m;
  }
  v4f acc[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) acc[f] = v4f{0, 0, 0, 0};
  const int whole = K / kScaleBlock;
  for (int j0 = wave; j0 < groups; j0 += kGemvWaves * AHEAD) {
    v4i w[AHEAD][2], x[AHEAD][MF][2];
    float sx[AHEAD][MF], sw[AHEAD];
    const int live = j0 + (AHEAD - 1) * kGemvWaves < whole ? AHEAD : 0;      // all blocks whole: no checks
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int j = j0 + u * kGemvWaves, jc = j < groups ? j : groups - 1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = jc * kScaleBlock + 16 * h;
        const bool in = live || (j < groups && k + 32 * lg < K);
#pragma unroll
        for (int f = 0; f < MF; ++f) x[u][f][h] = in ? *(const v4i*)(xp[f] + k) : v4i{0, 0, 0, 0};
      }
#pragma unroll
      for (int f = 0; f < MF; ++f) sx[u][f] = xs[f][(int64_t)jc * M];
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int j = j0 + u * kGemvWaves, jc = j < groups ? j : groups - 1;
      sw[u] = ws[jc];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = jc * kScaleBlock + 16 * h;
        w[u][h] = live || (j < groups && k + 32 * lg < K) ? *(const v4i*)(wp + k) : v4i{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const float sc = sw[u] * sx[u][f];
        const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join8(w[u][0], w[u][1]), join8(x[u][f][0], x[u][f][1]),
                                                                      v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[f][r] = __builtin_fmaf(sc, p[r], acc[f][r]);
      }
  }
  gemv_store<MF, YDT>(acc, part, wave, lane, M, N, n0, bias, y);
}

// Up to kFusedM tokens: the activations are quantized on the way, each wave
// its own blocks of K (16 consecutive features a lane, a block's maximum over 8
// lanes), through LDS into MFMA operands, while its weights are on their way:
// one launch and no workspace (4096 x 4096, one token: 4.4 us a call in a graph,
// 3.8 TB/s; quantized in a launch of its own 2.5 us more).
constexpr int kFusedM = 4;
template <int XDT, int YDT>
__global__ __launch_bounds__(kThreads) void k_gemv_block_fused(const void* __restrict__ x, int M, int K,
                                                               const uint8_t* __restrict__ wq,
                                                               const float* __restrict__ w_scale, int N,
                                                               const float* __restrict__ bias, void* __restrict__ y) {
  constexpr int AHEAD = 8;
  static_assert(AHEAD * 8 == 64, "a wave's lanes hold its blocks, 8 lanes a block");
  __shared__ v4f part[kGemvWaves][1][64];
  __shared__ __attribute__((aligned(16))) uint8_t codes[kGemvWaves][kFusedM][AHEAD * kScaleBlock];
  __shared__ float scales[kGemvWaves][kFusedM][AHEAD];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int groups = (K + kScaleBlock - 1) / kScaleBlock;
  const int n = n0 + lr < N ? n0 + lr : N - 1;
  const uint8_t* const wp = wq + (int64_t)n * K + 32 * lg;
  const float* const ws = w_scale + (int64_t)(n0 / kScaleBlock) * groups;
  const int mr = lr < M ? lr : M - 1;
  v4f acc[1] = {v4f{0, 0, 0, 0}};
  for (int j0 = wave; j0 < groups; j0 += kGemvWaves * AHEAD) {
    // this lane's 16 features, of block lane / 8
    const int kx = (j0 + (lane >> 3) * kGemvWaves) * kScaleBlock + 16 * (lane & 7);
    const bool inx = kx < K;
    constexpr int kPieces = XDT == DT_F32 ? 4 : 2;
    v4i raw[kFusedM][kPieces];
#pragma unroll
    for (int m = 0; m < kFusedM; ++m)
      if (m < M) {
        const v4i* p = (const v4i*)((const char*)x + ((int64_t)m * K + (inx ? kx : 0)) * (XDT == DT_F32 ? 4 : 2));
#pragma unroll
        for (int c = 0; c < kPieces; ++c) raw[m][c] = p[c];
      }
    v4i w[AHEAD][2];
    float sw[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int j = j0 + u * kGemvWaves, jc = j < groups ? j : groups - 1;
      sw[u] = ws[jc];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = jc * kScaleBlock + 16 * h;
        w[u][h] = *(const v4i*)(wp + (k + 32 * lg < K ? k : -32 * lg));
      }
    }
#pragma unroll
    for (int m = 0; m < kFusedM; ++m)
      if (m < M) {
        float v[16];
#pragma unroll
        for (int c = 0; c < kPieces; ++c) Chunk<XDT>::decode(raw[m][c], v + c * Chunk<XDT>::kElems);
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          v[e] = inx ? v[e] : 0.0f;
          amax = amax_of(amax, v[e]);
        }
        // over the block's 8 lanes: pairs, pairs of pairs, the half-row's two quads
        int am = __float_as_int(fabsf(amax));
        am = bits_max(am, __builtin_amdgcn_update_dpp(0, am, 0xB1, 0xF, 0xF, false));
        am = bits_max(am, __builtin_amdgcn_update_dpp(0, am, 0x4E, 0xF, 0xF, false));
        am = bits_max(am, __builtin_amdgcn_update_dpp(0, am, 0x141, 0xF, 0xF, false));
        float s = __int_as_float(am) / kFp8Max;
        s = s < kEps ? kEps : s;
        const v2i lo = codes8<XDT>(v, s), hi = codes8<XDT>(v + 8, s);
        *(v4i*)&codes[wave][m][lane * 16] = v4i{lo[0], lo[1], hi[0], hi[1]};
        if ((lane & 7) == 0) scales[wave][m][lane >> 3] = s;
      }
    // (LDS of this wave only, which it reads after its own writes)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      // codes past K are zeros, so the weights there (of the row's start) add nothing
      const v4i* c = (const v4i*)&codes[wave][mr][u * kScaleBlock + 32 * lg];
      const float sc = sw[u] * scales[wave][mr][u];
      const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join8(w[u][0], w[u][1]), join8(c[0], c[1]),
                                                                     v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[0][r] = __builtin_fmaf(sc, p[r], acc[0][r]);
    }
  }
  gemv_store<1, YDT>(acc, part, wave, lane, M, N, n0, bias, y);
}

template <int YDT>
hipError_t launch_product(const uint8_t* xq, const float* xs, int M, int K, const uint8_t* wq, const float* ws, int N,
                          const float* bias, void* y, hipStream_t st) {
  auto tiles = [&](int64_t bm, int64_t bn) { return (unsigned)(((M + bm - 1) / bm) * ((N + bn - 1) / bn)); };
  // Times are a product's alone, K = 4096.  Straight into registers where few tokens
  // meet few weight rows (16 tokens: 6.2 against 9.7 us at 4096 rows, 10.1 against 10.2 at 8192 and
  // 18.7 against 10.9 at 14336; 32 tokens: 8.4 against 9.9; 48: 11.6 against 10.1).
  if (M <= 32 && N < 8192) {
    const unsigned grid = (unsigned)((N + 15) / 16);
    if (M <= 16) k_gemv_block<1, 8, YDT><<<grid, kThreads, 0, st>>>(xq, xs, M, K, wq, ws, N, bias, y);
    else k_gemv_block<2, 4, YDT><<<grid, kThreads, 0, st>>>(xq, xs, M, K, wq, ws, N, bias, y);
  } else if (tiles(64, 64) <= 512) {
    // as long as the chip holds all of them, two a CU (4096 columns: 18.0 against 18.6 us for 512
    // tokens, 24.6 against 18.5 for 576); 8 waves (4: 12.0 against 11.4 us at 512 x 2048)
    k_gemm_tiles<64, 64, 2, 4, 4, YDT><<<tiles(64, 64), 512, 0, st>>>(xq, xs, M, K, wq, ws, N, bias, y);
  } else if (tiles(256, 256) < 192) {
    // 59.6 against 62.2 us at 2816 x 4096 (176 tiles of 256), 76.0 against 64.6 at 1024 x 14336 (224)
    k_gemm_tiles<128, 128, 2, 4, 4, YDT><<<tiles(128, 128), 512, 0, st>>>(xq, xs, M, K, wq, ws, N, bias, y);
  } else {
    k_gemm_tiles<256, 256, 2, 4, 2, YDT><<<tiles(256, 256), 512, 0, st>>>(xq, xs, M, K, wq, ws, N, bias, y);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_weight_block(const void* w, int dt, int64_t N, int64_t K, uint8_t* wq, float* w_scale,
                                     hipStream_t st) {
  const unsigned grid = (unsigned)(((K + kScaleBlock - 1) / kScaleBlock) * ((N + kScaleBlock - 1) / kScaleBlock));
  switch (dt) {
    case DT_F32: k_quant_weight_block<DT_F32><<<grid, kThreads, 0, st>>>(w, N, K, wq, w_scale); break;
    case DT_F16: k_quant_weight_block<DT_F16><<<grid, kThreads, 0, st>>>(w, N, K, wq, w_scale); break;
    default: k_quant_weight_block<DT_BF16><<<grid, kThreads, 0, st>>>(w, N, K, wq, w_scale); break;
  }
  return hipGetLastError();
}

hipError_t launch_quant_act_block(const void* x, int dt, int64_t M, int64_t K, uint8_t* xq, float* x_scale,
                                  hipStream_t st) {
  const int groups = (int)((K + kScaleBlock - 1) / kScaleBlock);
  const unsigned grid = (unsigned)((M * groups + kThreads / 16 - 1) / (kThreads / 16));
  switch (dt) {
    case DT_F32: k_quant_act_block<DT_F32><<<grid, kThreads, 0, st>>>(x, M, K, groups, xq, x_scale); break;
    case DT_F16: k_quant_act_block<DT_F16><<<grid, kThreads, 0, st>>>(x, M, K, groups, xq, x_scale); break;
    default: k_quant_act_block<DT_BF16><<<grid, kThreads, 0, st>>>(x, M, K, groups, xq, x_scale); break;
  }
  return hipGetLastError();
}

hipError_t launch_gemm_fp8_block(const uint8_t* xq, const float* x_scale, int64_t M, int64_t K, const uint8_t* wq,
                                 const float* w_scale, int64_t N, const float* bias, void* y, int ydt, hipStream_t st) {
  if (ydt == DT_F16) return launch_product<DT_F16>(xq, x_scale, (int)M, (int)K, wq, w_scale, (int)N, bias, y, st);
  return launch_product<DT_BF16>(xq, x_scale, (int)M, (int)K, wq, w_scale, (int)N, bias, y, st);
}

namespace {
template <int XDT>
hipError_t launch_fused(const void* x, int M, int K, const uint8_t* wq, const float* ws, int N, const float* bias, void* y,
                        int ydt, hipStream_t st) {
  const unsigned grid = (unsigned)((N + 15) / 16);
  if (ydt == DT_F16) k_gemv_block_fused<XDT, DT_F16><<<grid, kThreads, 0, st>>>(x, M, K, wq, ws, N, bias, y);
  else k_gemv_block_fused<XDT, DT_BF16><<<grid, kThreads, 0, st>>>(x, M, K, wq, ws, N, bias, y);
  return hipGetLastError();
}
}  // namespace

bool fp8_block_is_fused(int64_t M) { return M <= kFusedM; }

hipError_t launch_gemv_fp8_block(const void* x, int xdt, int64_t M, int64_t K, const uint8_t* wq, const float* w_scale,
                                 int64_t N, const float* bias, void* y, int ydt, hipStream_t st) {
  switch (xdt) {
    case DT_F32: return launch_fused<DT_F32>(x, (int)M, (int)K, wq, w_scale, (int)N, bias, y, ydt, st);
    case DT_F16: return launch_fused<DT_F16>(x, (int)M, (int)K, wq, w_scale, (int)N, bias, y, ydt, st);
    default: return launch_fused<DT_BF16>(x, (int)M, (int)K, wq, w_scale, (int)N, bias, y, ydt, st);
  }
}

}  // namespace q8
