// Backward passes of the fused linear layers (frozen packed weights):
//   dZ = dY * act'(Z)                          (gated: dG and dU from dH, G, U)
//   dbias = sum over rows of dZ
//   dX = add + s * sum over layers of dZ . D,  D[n][k] = (q - z) * scale
//
// The product contracts over N, the packed layout is made for contracting over
// K: a lane's code word is 8 columns of one row, but the B operand of dZ . D
// needs 8 rows of one column.  Transposing in the kernel costs either LDS
// traffic for the dequantized tile (as much again as the A operand's, which
// would bound the kernel by LDS) or byte shuffles in every workgroup that reads
// the weight.  The weights never change in training, so they are transposed
// once (transpose_codes_kernel): tiles of 16 input features x 128 output rows,
// whose words are B operands again.  The scale and zero point now vary along the
// contraction; they are the same for the 128 input features of a quantization
// group, so a workgroup's share is 4 bytes per row and group, staged in LDS.
#include <algorithm>

#include "epilogue.h"
#include "w4a16_device.h"
#include "w4a16_internal.h"

namespace w4a16 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

constexpr int kRsrcWord3 = 0x00020000;  // raw buffer resource, 32-bit data format
constexpr int kMetaBytes = 512;         // metadata of 128 rows and one quantization group
constexpr int kOutOfRange = 0x7ffffff0; // a buffer offset past every resource: loads read 0

__device__ __forceinline__ int uniform_int(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(mask), "v"(bits));
  return r;
}

// ---- transposed weights -----------------------------------------------------------

// One thread per 8 codes of the transposed layout: rows n0 .. n0 + 7 of input
// feature k.  Offline, so the 8 gathered bytes per thread are left to the caches.
template <bool W8>
__global__ __launch_bounds__(256) void transpose_codes_kernel(const uint8_t *Wq, int N, int K,
                                                              long long octets, uint8_t *Wt) {
  const long long o = (long long)blockIdx.x * 256 + threadIdx.x;
  if (o >= octets) return;
  const int t = (int)(o & 3), lane = (int)(o >> 2) & 63, c = lane >> 4, r = lane & 15;
  const int KB = K / kTileRows, NB = N / kTileRows;
  const int tile = (int)(o >> 8), g = tile / KB, b = tile - g * KB;
  const int k = b * kTileRows + r, n0 = g * kGroup + 32 * t + 8 * c;
  const int gk = k / kGroup, kk = k % kGroup, ts = kk / 32, cs = kk % 32 / 8, js = kk % 8;
  const int slot = js / 2 + 4 * (js % 2);
  uint32_t code[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (n0 < N) {  // N is a multiple of 16: all 8 rows or none
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int n = n0 + j;
      const size_t lane16 = ((size_t)gk * NB + n / kTileRows) * kWave + 16 * cs + n % kTileRows;
      code[j] = W8 ? Wq[lane16 * 32 + 8 * ts + js]
                   : (Wq[lane16 * 16 + 4 * ts + slot / 2] >> (4 * (slot & 1))) & 15u;
    }
  }
  if (W8) {
    uint32_t *dst = reinterpret_cast<uint32_t *>(Wt) + 2 * o;
    dst[0] = code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24;
    dst[1] = code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24;
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= code[2 * (i % 4) + i / 4] << (4 * i);
    reinterpret_cast<uint32_t *>(Wt)[o] = w;
  }
}

// One thread per (128-row group g, quantization group u, row j): its scale and
// its zero point plus the bias of the code's decoding, 1024 (or 64 for the codes
// that are decoded from the upper 4 bits of a byte), both exact in fp16.
template <bool W8>
__global__ __launch_bounds__(256) void transpose_meta_kernel(const _Float16 *scales,
                                                             const _Float16 *zeros, int N, int G,
                                                             long long count, uint8_t *meta) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= count) return;
  const int j = (int)(i & (kGroup - 1));
  const long long gu = i / kGroup;
  const int g = (int)(gu / G), u = (int)(gu - (long long)g * G), n = g * kGroup + j;
  _Float16 sc = (_Float16)0.f, z = (_Float16)0.f;
  if (n < N) {
    const size_t at = meta_index(n, u, N / kTileRows);
    sc = scales[at];
    z = zeros[at];
  }
  _Float16 *dst = reinterpret_cast<_Float16 *>(meta + gu * kMetaBytes);
  dst[j] = sc;
  dst[kGroup + j] = z + (_Float16)(!W8 && (j & 2) ? 64.f : 1024.f);
}

// ---- gradients of the epilogues -----------------------------------------------------

// dZ (gated: dG and dU) of a strip of rows, 8 columns per thread, and the
// strip's column sums: each thread sums its rows in order, then the row lanes
// meet in LDS, so the sums do not depend on scheduling.
// Bound by HBM: one read of dY and the pre-activations, one write of dZ.
// COLS columns per workgroup, 2048 / COLS rows at a time: 512 and 4, or, for
// column sums of few rows (one_strip), 32 and 64, where one strip is all
// rows and its sums are the result: no partial sums and no second launch.
constexpr int kGradCols = 512, kOneStripCols = 32;
struct GradArgs {
  const void *dY, *z, *u;      // z, u: pre-activations (null: dZ = dY, not written)
  void *dz, *du;
  float *part, *part2;         // column sums [strips][N] (null: not wanted)
  int M, N, rows, col_blocks;  // rows per strip
  int act;
};

template <bool BF, bool GATED, int COLS>
__global__ __launch_bounds__(256) void grad_kernel(GradArgs a) {
  constexpr int kAcross = COLS / 8, kRows = 256 / kAcross;  // threads along a row, rows at a time
  constexpr int kParts = COLS < 256 ? 256 / COLS : 1;       // of the rows, in the sum over row lanes
  const int strip = (int)blockIdx.x / a.col_blocks;
  const int col0 = ((int)blockIdx.x - strip * a.col_blocks) * COLS;
  const int x8 = (int)threadIdx.x % kAcross * 8, n = col0 + x8;
  const int lane_row = threadIdx.x / kAcross;
  const int m1 = min(a.M, (strip + 1) * a.rows);
  float s0[8] = {0, 0, 0, 0, 0, 0, 0, 0}, s1[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (n < a.N && !GATED && !a.dz) {  // column sums alone: up to eight loads in flight
    constexpr int kAtOnce = 8;
    for (int m = strip * a.rows + lane_row; m < m1; m += kAtOnce * kRows) {
      u32x4 d[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        d[k] = u32x4{0, 0, 0, 0};
        if (m + k * kRows < m1)
          d[k] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.dY) +
                                                  (size_t)(m + k * kRows) * a.N + n);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) s0[j] += act_to_f32<BF>((uint16_t)(d[k][j / 2] >> (16 * (j & 1))));
    }
  } else if (n < a.N) {
#pragma unroll 2
    for (int m = strip * a.rows + lane_row; m < m1; m += kRows) {
      const size_t at = (size_t)m * a.N + n;
      const u32x4 d = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.dY) + at);
      u32x4 u = d, oz, ou;
      const u32x4 z = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.z) + at);
      if (GATED) u = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.u) + at);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t wz = 0, wu = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float dy = act_to_f32<BF>((uint16_t)(d[q] >> (16 * h)));
          const float zv = act_to_f32<BF>((uint16_t)(z[q] >> (16 * h)));
          float dz = dy * act_grad(zv, a.act);
          if (GATED) {
            const float du = dy * act_value(zv, a.act);
            dz *= act_to_f32<BF>((uint16_t)(u[q] >> (16 * h)));
            s1[2 * q + h] += du;
            wu |= (uint32_t)f32_to_act<BF>(du) << (16 * h);
          }
          s0[2 * q + h] += dz;
          wz |= (uint32_t)f32_to_act<BF>(dz) << (16 * h);
        }
        oz[q] = wz;
        ou[q] = wu;
      }
      *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.dz) + at) = oz;
      if (GATED) *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.du) + at) = ou;
    }
  }
  __shared__ float red[kRows][COLS];
  auto column_sums = [&](const float (&s)[8], float *part) {
    if (!part) return;  // uniform
#pragma unroll
    for (int j = 0; j < 8; ++j) red[lane_row][x8 + j] = s[j];
    __syncthreads();
    if constexpr (kParts > 1) {  // kRows / kParts rows each, in order, into the first of them
      const int x = (int)threadIdx.x % COLS, i0 = (int)threadIdx.x / COLS * (kRows / kParts);
      float sum = red[i0][x];
#pragma unroll
      for (int i = 1; i < kRows / kParts; ++i) sum += red[i0 + i][x];
      red[i0][x] = sum;
      __syncthreads();
    }
    for (int x = threadIdx.x; x < COLS; x += 256) {
      float sum;
      if constexpr (kRows == 4) {
        sum = (red[0][x] + red[1][x]) + (red[2][x] + red[3][x]);
      } else {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kRows; i += kRows / kParts) sum += red[i][x];
      }
      if (col0 + x < a.N) part[(size_t)strip * a.N + col0 + x] = sum;
    }
    __syncthreads();
  };
  column_sums(s0, a.part);
  if (GATED) column_sums(s1, a.part2);
}

// out[n] = the strips' sums (0 without strips): 8 lanes per column, each over
// every 8th strip, then the lanes in order.  (One thread per column, one load
// after the other, took 13 us for 50 strips of 3584 columns.)
__global__ __launch_bounds__(256) void bias_kernel(const float *part, int strips, int N, float *out) {
  const int x = threadIdx.x & 31, lane = threadIdx.x >> 5;
  const int n = (int)blockIdx.x * 32 + x;
  float s = 0.f;
  if (n < N) {
#pragma unroll 4
    for (int k = lane; k < strips; k += 8) s += part[(size_t)k * N + n];
  }
  __shared__ float red[8][32];
  red[lane][x] = s;
  __syncthreads();
  if (lane == 0 && n < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][x];
    out[n] = s;
  }
}

// ---- dX ------------------------------------------------------------------------------

struct DxTerm {
  const void *dZ;       // [M][N]
  const uint8_t *Wt, *meta;
  int N, stage0;        // stage0: stages (128 rows of N each) of the terms before
};
struct DxArgs {
  DxTerm t[kMaxDxTerms];
  int count;
  const _Float16 *s;
  const void *add;
  void *dX;
  float *part;          // split > 1: split fp32 [M][K] partial slabs
  int M, K;
  int tiles_k, tiles;   // output blocks along K, and in all
  int split, stages;
};

// dX block of 16 TM x 64 TN, four waves of 16 TM x 16 TN, in stages of 128 rows
// of one term's N:
//   * dZ's rows go from memory into LDS with DMA loads, double-buffered, one
//     barrier per stage, 16-byte chunks XOR-swizzled by the row so that the A
//     operand reads of 16 rows hit distinct banks; chunks past N read zeros;
//   * the stage's scales and zero points (1 KB for 256 columns) follow the same
//     way; a k step's 8 rows are one 16-byte read each, shared by the 16 lanes;
//   * the wave's code tiles (its B operands) are loaded into registers one
//     stage ahead, in two register sets that alternate.
// A weight's dequantization: (q - z) exact in fp16, times the scale, rounded
// once to fp16; bf16 takes the product in fp32 (v_fma_mix, exact: 8 + 11 bits)
// and rounds it once: 5 instructions for two weights, where converting code
// and scale to fp32 first would take 7.  Both operands are rounded to the
// activations' type because the MFMA takes 16-bit ones: dZ as it is stored, and D
// with its scale, which varies along the contraction here and so cannot
// multiply the fp32 sums instead.
// N is split across workgroups when the output blocks leave CUs idle: fp32
// partials, added in a fixed order by dx_reduce_kernel.
// KS = 2: two slices of four waves each walk every other stage of the
// workgroup's range into LDS stages of their own, and the sums meet through
// LDS at the end (slice 0's plus slice 1's): two waves per SIMD without fp32
// partials in memory.
template <int TM, int TN, int KS, bool BF, bool W8>
__global__ __launch_bounds__(256 * KS) __attribute__((amdgpu_waves_per_eu(TN == 2 ? 4 : 2, TN == 2 ? 4 : 2))) void dx_kernel(
    DxArgs P) {
  constexpr int kCW = W8 ? 2 : 1;  // 16-byte code pieces per lane per tile
  constexpr int BM = TM * 16, BN = 64 * TN;
  constexpr int kRowChunks = kGroup / 8;  // 16-byte chunks per row per stage
  constexpr int kDma = TM;                // DMA loads per wave per stage
  static_assert(kDma * 4 * 64 == BM * kRowChunks, "a stage is whole DMA loads");
  static_assert(KS == 1 || BM * BN * 4 <= KS * 2 * BM * kGroup * 2, "the slices' sums fit the dZ stages");
  __shared__ __attribute__((aligned(16))) _Float16 As[KS][2][BM * kGroup];
  __shared__ __attribute__((aligned(16))) unsigned char Ms[KS][2][1024];

  const int M = P.M, K = P.K;
  const int tid = threadIdx.x, lane = tid & 63, wv = uniform_int(tid >> 6);
  const int ks = KS == 1 ? 0 : wv >> 2, wave = KS == 1 ? wv : wv & 3;  // slice; the wave's column
  const int c = lane >> 4, r = lane & 15;
  // Workgroups go to the eight XCDs round robin: a split launch is renumbered
  // so that each XCD takes a contiguous run of (split, block) pairs, which
  // share dZ rows and code panels in its L2.
  const int L = P.split * P.tiles, q8 = L >> 3, block = (int)blockIdx.x;
  const int local = (P.split > 1 && block < 8 * q8) ? (block & 7) * q8 + (block >> 3) : block;
  const int sp = local / P.tiles, t = local - sp * P.tiles;
  const int mt = t / P.tiles_k;
  const int k0 = (t - mt * P.tiles_k) * BN, m0 = mt * BM;
  const int KB = K / kTileRows, G = K / kGroup;
  const int sb = (int)((long long)P.stages * sp / P.split);
  const int se = (int)((long long)P.stages * (sp + 1) / P.split);
  const int rows = min(BM, M - m0);

  float4v acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = float4v{0.f, 0.f, 0.f, 0.f};

  for (int ti = 0; ti < P.count; ++ti) {
    const DxTerm &T = P.t[ti];
    const int N = T.N, NG = (N + kGroup - 1) / kGroup;
    const int gb = max(sb - T.stage0, 0), ge = min(se - T.stage0, NG);
    if (gb >= ge) continue;

    // dZ: wave load u fills LDS chunks p = (u * 4 + wave) * 64 + lane; chunk p is
    // row p / 16 = 16 u + 4 wave + lane / 16, physical chunk p % 16, holding
    // logical chunk lc = (p % 16) ^ (row % 16), the same for every u.  Rows past
    // M lie past the resource and read zeros, as do chunks past N.
    const __amdgpu_buffer_rsrc_t xrs = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(static_cast<const uint16_t *>(T.dZ) + (size_t)m0 * N), (short)0, rows * N * 2, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t wrs = __builtin_amdgcn_make_buffer_rsrc(
        (void *)T.Wt, (short)0, (int)min((size_t)0x7fffffff, (size_t)KB * NG * kTileBytes * kCW), kRsrcWord3);
    const __amdgpu_buffer_rsrc_t mrs = __builtin_amdgcn_make_buffer_rsrc(
        (void *)T.meta, (short)0, (int)min((size_t)0x7fffffff, (size_t)NG * G * kMetaBytes), kRsrcWord3);
    const int row0 = 4 * wave + (lane >> 4), lc = (lane & 15) ^ row0;
    const int xoff = (row0 * N + 8 * lc) * 2;
    // (left: columns of the stage that count, 0 for one past the range)
    auto load_x = [&](int g, int left, int buf) {
      const int vo = 8 * lc < left ? xoff : kOutOfRange;
#pragma unroll
      for (int u = 0; u < kDma; ++u) {
        const int vu = (int)((unsigned)vo + 32u * u * N);  // still out of range where vo is
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            xrs, (__attribute__((address_space(3))) void *)(&As[ks][buf][(u * 4 + wave) * 64 * 8]), 16,
            vu, g * kGroup * 2, 0, 0);
      }
      // scales and zero points of the block's quantization groups: 256 bytes a wave
      const int mo = (wave * 64 + lane) * 4;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          mrs, (__attribute__((address_space(3))) void *)(&Ms[ks][buf][wave * 256]), 4, mo,
          (g * G + k0 / kGroup) * kMetaBytes, 0, 0);
    };
    const int kb0 = k0 / kTileRows + wave * TN;
    const int tile_stride = KB * kTileBytes * kCW;
    struct BStage {
      u32x4 code[TN][kCW];
    };
    // column blocks past K re-read the last one (never stored)
    auto load_b = [&](int g, BStage &b) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int kb = min(kb0 + j, KB - 1);
#pragma unroll
        for (int h = 0; h < kCW; ++h)
          b.code[j][h] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(wrs, (kb * 64 + lane) * 16 * kCW + 16 * h,
                                                           g * tile_stride, 0));
      }
    };
    // the wave's quantization group among the block's
    const int ul = (wave * TN * kTileRows) / kGroup;

    // A operands of one k step; small tiles have registers to read them a k step
    // ahead, the first before the next stage's loads are issued
    constexpr bool kAhead = TN == 2;
    auto read_a = [&](int tt, int buf, u32x4 (&a)[TM]) {
      const int pc = (4 * tt + c) ^ r;
#pragma unroll
      for (int i = 0; i < TM; ++i)
        a[i] = *reinterpret_cast<const u32x4 *>(&As[ks][buf][(16 * i + r) * kGroup + 8 * pc]);
    };
    auto compute = [&](const BStage &b, int buf, u32x4 (&a)[TM]) {
      const _Float16 *ms = reinterpret_cast<const _Float16 *>(&Ms[ks][buf][ul * kMetaBytes]) + 8 * c;
      struct Meta {
        half8 scale, bias;
      };
      auto meta_at = [&](int tt) -> Meta {
        return {*reinterpret_cast<const half8 *>(ms + 32 * tt),
                *reinterpret_cast<const half8 *>(ms + kGroup + 32 * tt)};
      };
      auto dequant = [&](int j, int tt, const Meta &mt8) -> u32x4 {
        half2v e[4];
        if constexpr (W8) {
          const uint32_t wa = b.code[j][tt >> 1][2 * (tt & 1)], wb = b.code[j][tt >> 1][2 * (tt & 1) + 1];
          const uint32_t magic = 0x64646464u;
          e[0] = as_half2(__builtin_amdgcn_perm(magic, wa, 0x05010400u));
          e[1] = as_half2(__builtin_amdgcn_perm(magic, wa, 0x05030402u));
          e[2] = as_half2(__builtin_amdgcn_perm(magic, wb, 0x05010400u));
          e[3] = as_half2(__builtin_amdgcn_perm(magic, wb, 0x05030402u));
        } else {
          const uint32_t w = b.code[j][0][tt], w8 = w >> 8;
          const half2v sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
          e[0] = as_half2(and_or(w, 0x000F000Fu, kMagic2));
          e[1] = as_half2(and_or(w, 0x00F000F0u, kMagic2)) * sixteenth;
          e[2] = as_half2(and_or(w8, 0x000F000Fu, kMagic2));
          e[3] = as_half2(and_or(w8, 0x00F000F0u, kMagic2)) * sixteenth;
        }
        u32x4 out;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const half2v bias = {mt8.bias[2 * p], mt8.bias[2 * p + 1]};
          const half2v scale = {mt8.scale[2 * p], mt8.scale[2 * p + 1]};
          const half2v v = e[p] - bias;  // q - z, exact
          if constexpr (BF)
            out[p] = pack_bf16x2(__builtin_fmaf((float)v[0], (float)scale[0], 0.f),
                                 __builtin_fmaf((float)v[1], (float)scale[1], 0.f));
          else
            out[p] = __builtin_bit_cast(uint32_t, v * scale);
        }
        return out;
      };
      // software pipeline: k step tt + 1's B operands are dequantized while k
      // step tt's MFMAs run
      u32x4 bop[TN];
      Meta m = meta_at(0);
#pragma unroll
      for (int j = 0; j < TN; ++j) bop[j] = dequant(j, 0, m);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        u32x4 bnx[TN];
        if (tt < 3) {
          m = meta_at(tt + 1);
#pragma unroll
          for (int j = 0; j < TN; ++j) bnx[j] = dequant(j, tt + 1, m);
        }
        u32x4 anx[TM];
        if (kAhead && tt < 3) read_a(tt + 1, buf, anx);
        const int pc = (4 * tt + c) ^ r;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const u32x4 aop = kAhead ? a[i] : *reinterpret_cast<const u32x4 *>(
                                                &As[ks][buf][(16 * i + r) * kGroup + 8 * pc]);
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = BF ? mfma16_bf16(aop, bop[j], acc[i][j])
                           : mfma16(__builtin_bit_cast(half8, aop), __builtin_bit_cast(half8, bop[j]),
                                    acc[i][j]);
        }
        if (tt < 3) {
          if (kAhead) {
#pragma unroll
            for (int i = 0; i < TM; ++i) a[i] = anx[i];
          }
#pragma unroll
          for (int j = 0; j < TN; ++j) bop[j] = bnx[j];
        }
      }
    };

    // one stage per step, as in the forward kernel: wait for this stage's loads
    // (issued a step ago) and for every wave to be past the step before, issue
    // the next stage's, compute.  Past the range the loads re-read its last
    // stage into buffers and registers that nobody reads.
    BStage b0, b1;
    // stage i of this slice; every slice runs the same number of steps (and
    // barriers), and one past the range adds zeros: its dZ is read as zeros
    const int nsteps = (ge - gb + KS - 1) / KS;
    auto load_stage = [&](int i, BStage &b, int buf) {
      const int g = gb + ks + min(i, nsteps - 1) * KS, gc = KS == 1 ? g : min(g, ge - 1);
      load_x(gc, KS == 1 || g < ge ? N - g * kGroup : 0, buf);
      load_b(gc, b);
    };
    auto step = [&](int i, BStage &cur, BStage &nxt, int buf) {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      u32x4 a[TM];
      if (kAhead) read_a(0, buf, a);
      load_stage(i + 1, nxt, buf ^ 1);
      compute(cur, buf, a);
    };
    // the term before may still be read, and its last loads still land, in LDS
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    load_stage(0, b0, 0);
    for (int i = 0; i < nsteps; i += 2) {
      step(i, b0, b1, 0);
      if (i + 1 < nsteps) step(i + 1, b1, b0, 1);
    }
  }
  // the last step's DMA must land before the workgroup's LDS is released
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if constexpr (KS == 2) {
    float *red = reinterpret_cast<float *>(&As[0][0][0]);
    __syncthreads();  // every wave is done with the dZ stages
    if (ks == 1) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          *reinterpret_cast<float4v *>(&red[((i * TN + j) * 4 + wave) * 256 + lane * 4]) = acc[i][j];
    }
    __syncthreads();
    if (ks == 1) return;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] += *reinterpret_cast<const float4v *>(&red[((i * TN + j) * 4 + wave) * 256 + lane * 4]);
  }

  // lane holds D[4c + v][r] of each 16x16 sub-block.  Buffer resources that
  // start at the sub-block's first row and end at row M drop rows past M; a
  // 16-column block lies inside K as a whole or not at all.
  const int kb0 = k0 / kTileRows + wave * TN;
  float sv[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j)
    sv[j] = P.s && kb0 + j < KB ? (float)P.s[(kb0 + j) * kTileRows + r] : 1.f;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int mi = m0 + 16 * i;
    if (mi >= M) break;
    const int n16 = min(M - mi, 16);
    auto rsrc = [&](const void *p, size_t row0, int esize) {
      return __builtin_amdgcn_make_buffer_rsrc(
          (void *)(static_cast<const char *>(p) + row0 * K * esize), (short)0, n16 * K * esize, kRsrcWord3);
    };
    auto at = [&](int j, int v) { return (4 * c + v) * K + (kb0 + j) * kTileRows + r; };
    if (P.split > 1) {
      const __amdgpu_buffer_rsrc_t prs = rsrc(P.part, (size_t)sp * M + mi, 4);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        if (kb0 + j >= KB) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float x = acc[i][j][v];  // (a bit cast of the vector element itself takes element 0)
          __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), prs, at(j, v) * 4, 0, 0);
        }
      }
      continue;
    }
    uint16_t add[TN][4];
    if (P.add) {
      const __amdgpu_buffer_rsrc_t ars = rsrc(P.add, mi, 2);
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          add[j][v] = __builtin_amdgcn_raw_buffer_load_b16(ars, kb0 + j < KB ? at(j, v) * 2 : 0, 0, 0);
    }
    const __amdgpu_buffer_rsrc_t yrs = rsrc(P.dX, mi, 2);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if (kb0 + j >= KB) continue;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float x = acc[i][j][v] * sv[j];
        if (P.add) x += act_to_f32<BF>(add[j][v]);
        __builtin_amdgcn_raw_buffer_store_b16(f32_to_act<BF>(x), yrs, at(j, v) * 2, 0, 0);
      }
    }
  }
}

// dX from the split partials, in split order; four outputs of one row per thread.
template <bool BF>
__global__ __launch_bounds__(256) void dx_reduce_kernel(DxArgs P) {
  const long long quads = (long long)P.M * P.K / 4;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  float4v x = sum_partials(reinterpret_cast<const float4v *>(P.part) + i, quads, P.split);
  typedef _Float16 half4 __attribute__((ext_vector_type(4)));
  if (P.s) {
    const half4 s = *reinterpret_cast<const half4 *>(P.s + (i * 4) % P.K);
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] *= (float)s[v];
  }
  u16x4 out;
  if (P.add) {
    const u16x4 a = reinterpret_cast<const u16x4 *>(P.add)[i];
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] += act_to_f32<BF>(a[v]);
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) out[v] = f32_to_act<BF>(x[v]);
  reinterpret_cast<u16x4 *>(P.dX)[i] = out;
}

// ---- plans and launches ----------------------------------------------------------------

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Column sums of few rows: one strip, without a second launch.  One limit for every
// width and activation, below each of their crossovers.  Measured in us per call
// (bf16), strips against one, with 14336 columns: no activation, M = 200 6.5 and 3.9,
// M = 256 6.6 and 4.3; SiLU, M = 128 6.8 and 5.3, M = 256 8.4 and 7.8; gated, M = 64
// 9.7 and 5.2, M = 256 13.8 and 11.9.  At the limit one strip is 0.2-2.8 us ahead in
// all nine sweeps (4096, 14336 and 18944 columns; M = 200 of 18944 SiLU columns alone is
// behind, 9.7 against 9.4).  Past it the sides part: no activation, 4096 columns,
// M = 1024 6.5 and 5.2, 14336 columns, M = 512 6.8 and 6.4, 18944 columns 7.5 and 8.2;
// SiLU, 4096 columns, M = 384 7.0 and 8.1, 14336 columns 10.7 and 10.2; gated, 18944
// columns, M = 384 20.5 and 23.3.  The one limit leaves up to 2.8 us there (plain sums
// of 4096 columns, M = 384: 6.9 and 4.0).
bool one_strip(int M, bool sums) { return sums && M <= 256; }

// Rows per strip of grad_kernel: 32, fewer while the launch has under 512
// workgroups (each is 256 threads: two per CU), more where column sums are
// wanted and 256 strips would not cover M (their partials stay below 1/128 of
// what the kernel reads).
int strip_rows(int M, int N, bool sums) {
  const long long cols = (N + kGradCols - 1) / kGradCols;
  int rows = 32;
  while (rows > 4 && cols * ((M + rows - 1) / rows) < 512) rows /= 2;
  if (sums) rows = std::max(rows, ((M + 255) / 256 + 3) / 4 * 4);
  return rows;
}
int strips_of(int M, int N, bool sums) {
  const int rows = strip_rows(M, N, sums);
  return (M + rows - 1) / rows;
}

struct DxPlan {
  int tm, tn, ks, split, stages;
  long long tiles;
};
// A block shape and its time per step (ks stages) with one and with two
// workgroups on a CU, in us (measured with bf16 activations and INT4 codes).
struct DxShape {
  int tm, tn, ks;
  double one, two;
};
constexpr int kDxMaxSplit = 32;

// Blocks of 128 x 256 (96 x 256 for INT8 codes, whose registers do not allow
// 128) for large products; 64 x 128 or 48 x 128 (32 x 128 and 16 x 128 where
// those cover M), with two slices per workgroup, where those would leave CUs idle.  The
// stages are split across workgroups (fp32 partials) and the shape is chosen by
// a model of the launch: rounds of at most two workgroups per CU, each as long
// as its steps, plus the partials' traffic and the second launch.  Measured, in
// us: M = 2048, N = 14336, K = 4096: 128 x 256 split in two 211, 64 x 128 289;
// M = 200, N = K = 3584: 128 x 256 split in four 27.2, 64 x 128 split in two
// 16.7 (one slice: 17.4); M = 64, N = 2 x 14336, K = 4096: 42.6 and 29.2 (34.4).
DxPlan plan_dx(const DxDesc &d) {
  static const DxShape large = {8, 4, 1, 2.9, 3.5}, large8 = {6, 4, 1, 2.5, 3.1};
  static const DxShape s64 = {4, 2, 2, 1.55, 2.65}, s48 = {3, 2, 2, 1.45, 2.4};
  static const DxShape s32 = {2, 2, 2, 1.3, 2.4}, s16 = {1, 2, 2, 1.2, 2.2};
  DxPlan best = {};
  double best_us = 0.0;
  int stages = 0;
  for (int i = 0; i < d.count; ++i) stages += (d.N[i] + kGroup - 1) / kGroup;
  const DxShape *const small = d.M > 32 ? &s64 : d.M > 16 ? &s32 : &s16;
  const DxShape *const shapes[3] = {small, d.M > 32 ? &s48 : nullptr,
                                    d.M > 64 ? (d.w8 ? &large8 : &large) : nullptr};
  for (const DxShape *s : shapes) {
    if (!s) continue;
    const long long tiles =
        (long long)((d.K + 64 * s->tn - 1) / (64 * s->tn)) * ((d.M + 16 * s->tm - 1) / (16 * s->tm));
    for (int split = 1; split <= kDxMaxSplit && split <= stages; ++split) {
      const long long wgs = tiles * split, rest = wgs % 512;
      const double rounds = (double)(wgs / 512) * s->two + (rest == 0 ? 0.0 : rest <= 256 ? s->one : s->two);
      const int steps = ((stages + split - 1) / split + s->ks - 1) / s->ks;
      const double mk = (double)d.M * d.K;
      const double us = rounds * (steps + 0.5) +
                        (split > 1 ? 2.5 + (4 * split + 2) * mk / 4.5e6 + (4 * split - 2) * mk / 9.0e6 : 0.0);
      if (best.split == 0 || us < best_us) {
        best_us = us;
        best = {s->tm, s->tn, s->ks, split, stages, tiles};
      }
    }
  }
  return best;
}

template <bool BF, bool W8>
void launch_dx_tile(const DxPlan &p, dim3 grid, hipStream_t stream, const DxArgs &a) {
#define W4_DX(TM, TN, KS)                                                                        \
  if (p.tm == TM && p.tn == TN && p.ks == KS)                                                    \
  hipLaunchKernelGGL((dx_kernel<TM, TN, KS, BF, W8>), grid, dim3(256 * KS), 0, stream, a)
  W4_DX((W8 ? 6 : 8), 4, 1);
  W4_DX(4, 2, 2);
  W4_DX(3, 2, 2);
  W4_DX(2, 2, 2);
  W4_DX(1, 2, 2);
#undef W4_DX
}

}  // namespace

hipError_t launch_transpose(const void *Wq, const void *scales, const void *zeros, int N, int K,
                            bool w8, void *Wt, void *meta, hipStream_t stream) {
  const int NG = (N + kGroup - 1) / kGroup, G = K / kGroup;
  const long long octets = (long long)K * NG * (kGroup / 8), rows = (long long)NG * G * kGroup;
  const dim3 cg((unsigned)((octets + 255) / 256)), mg((unsigned)((rows + 255) / 256)), th(256);
  const uint8_t *q = static_cast<const uint8_t *>(Wq);
  const _Float16 *s = static_cast<const _Float16 *>(scales), *z = static_cast<const _Float16 *>(zeros);
  if (w8) {
    hipLaunchKernelGGL(transpose_codes_kernel<true>, cg, th, 0, stream, q, N, K, octets, static_cast<uint8_t *>(Wt));
    hipLaunchKernelGGL(transpose_meta_kernel<true>, mg, th, 0, stream, s, z, N, G, rows, static_cast<uint8_t *>(meta));
  } else {
    hipLaunchKernelGGL(transpose_codes_kernel<false>, cg, th, 0, stream, q, N, K, octets, static_cast<uint8_t *>(Wt));
    hipLaunchKernelGGL(transpose_meta_kernel<false>, mg, th, 0, stream, s, z, N, G, rows, static_cast<uint8_t *>(meta));
  }
  return hipGetLastError();
}

size_t grad_workspace_bytes(int M, int N, int sums) {
  if (!sums || one_strip(M, true)) return 0;
  return sums * align256((size_t)strips_of(M, N, true) * N * sizeof(float));
}

hipError_t launch_grad(const GradDesc &d, void *workspace, hipStream_t stream) {
  const bool gated = d.u != nullptr, sums = d.db || d.db2;
  const bool one = d.M > 0 && one_strip(d.M, sums);
  const int strips = d.M == 0 ? 0 : one ? 1 : strips_of(d.M, d.N, sums);
  GradArgs a = {d.dY, d.z, d.u, d.dz, d.du, nullptr, nullptr, d.M, d.N, 0, 0, d.act};
  char *ws = static_cast<char *>(workspace);
  const size_t slab = align256((size_t)strips * d.N * sizeof(float));
  if (one) {
    a.part = static_cast<float *>(d.db);
    a.part2 = static_cast<float *>(d.db2);
  } else {
    if (d.db) {
      a.part = reinterpret_cast<float *>(ws);
      ws += slab;
    }
    if (d.db2) a.part2 = reinterpret_cast<float *>(ws);
  }
  if (strips > 0) {
    a.rows = one ? d.M : strip_rows(d.M, d.N, sums);
    const int cols = one ? kOneStripCols : kGradCols;
    a.col_blocks = (d.N + cols - 1) / cols;
    const dim3 grid((unsigned)(strips * (long long)a.col_blocks)), th(256);
#define W4_GRAD(BF, GATED)                                                                       \
  if (d.bf16 == BF && gated == GATED) {                                                          \
    if (one)                                                                                     \
      hipLaunchKernelGGL((grad_kernel<BF, GATED, kOneStripCols>), grid, th, 0, stream, a);       \
    else                                                                                         \
      hipLaunchKernelGGL((grad_kernel<BF, GATED, kGradCols>), grid, th, 0, stream, a);           \
  }
    W4_GRAD(true, true)
    W4_GRAD(true, false)
    W4_GRAD(false, true)
    W4_GRAD(false, false)
#undef W4_GRAD
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || one) return e;
  }
  const dim3 bg((unsigned)((d.N + 31) / 32)), th(256);
  if (d.db) hipLaunchKernelGGL(bias_kernel, bg, th, 0, stream, a.part, strips, d.N, static_cast<float *>(d.db));
  if (d.db2) hipLaunchKernelGGL(bias_kernel, bg, th, 0, stream, a.part2, strips, d.N, static_cast<float *>(d.db2));
  return hipGetLastError();
}

size_t dx_workspace_bytes(const DxDesc &d) {
  const DxPlan p = plan_dx(d);
  return p.split > 1 ? (size_t)p.split * d.M * d.K * sizeof(float) : 0;
}

hipError_t launch_dx(const DxDesc &d, void *workspace, hipStream_t stream) {
  if (d.count < 1 || d.count > kMaxDxTerms || d.M < 1) return hipErrorInvalidValue;
  const DxPlan p = plan_dx(d);
  if (p.tiles * p.split > INT32_MAX) return hipErrorInvalidValue;
  DxArgs a = {};
  int stage0 = 0;
  for (int i = 0; i < d.count; ++i) {
    a.t[i] = {d.dZ[i], static_cast<const uint8_t *>(d.Wt[i]), static_cast<const uint8_t *>(d.meta[i]),
              d.N[i], stage0};
    stage0 += (d.N[i] + kGroup - 1) / kGroup;
  }
  a.count = d.count;
  a.s = static_cast<const _Float16 *>(d.s);
  a.add = d.add;
  a.dX = d.dX;
  a.part = p.split > 1 ? static_cast<float *>(workspace) : nullptr;
  a.M = d.M;
  a.K = d.K;
  a.tiles_k = (d.K + 64 * p.tn - 1) / (64 * p.tn);
  a.tiles = (int)p.tiles;
  a.split = p.split;
  a.stages = p.stages;
  const dim3 grid((unsigned)(p.tiles * p.split));
  if (d.bf16 && d.w8)
    launch_dx_tile<true, true>(p, grid, stream, a);
  else if (d.bf16)
    launch_dx_tile<true, false>(p, grid, stream, a);
  else if (d.w8)
    launch_dx_tile<false, true>(p, grid, stream, a);
  else
    launch_dx_tile<false, false>(p, grid, stream, a);
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && p.split > 1) {
    const dim3 rg((unsigned)(((long long)d.M * d.K / 4 + 255) / 256));
    if (d.bf16)
      hipLaunchKernelGGL(dx_reduce_kernel<true>, rg, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL(dx_reduce_kernel<false>, rg, dim3(256), 0, stream, a);
    err = hipGetLastError();
  }
  return err;
}

}  // namespace w4a16
