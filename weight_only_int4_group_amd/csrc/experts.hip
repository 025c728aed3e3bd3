// The experts' gated feed-forward blocks over packed INT4 weights, and their backward.
//
//   forward   G = X . Wg_e^T,  U = X . Wu_e^T,  H = act(G) * U * s_down,
//             Y = residual + sum over a token's slots of w * (H . Wd_e^T)
//   backward  dH = (dY . Wd_e) * s_down,  dw = <dH, act(G) * U>,
//             dG = w dH U act'(G),  dU = w dH act(G),
//             dX = add + s * sum over the slots of (dG . Wg_e + dU . Wu_e)
//
// A slot is one of a token's k choices.  plan_kernel sorts the slots by expert and cuts each
// expert's run into tiles of rows; a product's workgroup takes one tile and a strip of the
// expert's outputs.  How many tiles there are is known on the GPU alone: the grids cover
// the most there can be, and workgroups past the last tile end at once.  The order of an
// expert's rows is whatever the sort's atomics give; no result depends on it, since a
// row of a product does not depend on the rows beside it.
//
// Each slot's contribution to Y (or dX) is kept in fp32, weighted, in the slot's own row;
// combine_kernel adds a token's k rows in their order.  (Atomic adds into Y would save
// that pass, and give other bits every time.)
#include <algorithm>

#include "epilogue.h"
#include "w4a16_device.h"
#include "w4a16_internal.h"

namespace w4a16 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

constexpr int kRsrcWord3 = 0x00020000;  // raw buffer resource, 32-bit data format
constexpr int kMetaBytes = 512;         // transposed weights: metadata of 128 rows and one group
constexpr int kOutOfRange = 0x7ffffff0; // a buffer offset past every resource: loads read 0

__device__ __forceinline__ int uniform_int(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(mask), "s"(bits));
  return r;
}

template <bool BF>
__device__ __forceinline__ float4v mfma(u32x4 a, u32x4 b, float4v c) {
  if constexpr (BF)
    return mfma16_bf16(a, b, c);
  else
    return mfma16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c);
}

// Eight codes of one word as an exact MFMA operand, c + q with c = 128 (bf16) or 64
// (fp16): an OR into the mantissa of c, whose last bit that holds 1 lies at the
// bottom (bf16) or at bit 4 (fp16).  Seven instructions, and nothing rounded; with
// xs the sum of a row's activations over the group, its dot product with (q - z) is
// the MFMA's sum minus (c + z) xs, in fp32.
template <bool BF>
constexpr float kCodeBase = BF ? 128.f : 64.f;
// (No inline assembly here: an MFMA may read a register only two wait states after a
// vector instruction wrote it, and the compiler sees to that for its own instructions alone.)
// Part p of it: columns 2p and 2p + 1.
template <bool BF>
__device__ __forceinline__ uint32_t code_part(uint32_t w, int p) {
  constexpr uint32_t mask = BF ? 0x000F000Fu : 0x00F000F0u, base = BF ? kMagicBF : 0x54005400u;
  const uint32_t x = BF ? w >> (4 * p) : p ? w >> (4 * p - 4) : w << 4;
  // (x & mask) | base as one instruction (bit by bit, 0xEA is the truth table); written with
  // operators it becomes two
  return (uint32_t)__builtin_amdgcn_bitop3_b32(x, mask, base, 0xEA);
}
template <bool BF>
__device__ __forceinline__ u32x4 code_operand(uint32_t w) {
  return (u32x4){code_part<BF>(w, 0), code_part<BF>(w, 1), code_part<BF>(w, 2), code_part<BF>(w, 3)};
}
template <bool BF>
__device__ __forceinline__ u32x4 ones_operand() {
  const uint32_t one = BF ? 0x3F803F80u : 0x3C003C00u;
  return (u32x4){one, one, one, one};
}

// Eight codes of one word as fp16, exact: columns 2p and 2p + 1 in e[p], plus 1024 (p even) or
// 64 (p odd).
__device__ __forceinline__ void code_halves(uint32_t w, half2v (&e)[4]) {
  const uint32_t w8 = w >> 8;
  const half2v sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  e[0] = as_half2(and_or(w, 0x000F000Fu, kMagic2));
  e[1] = as_half2(and_or(w, 0x00F000F0u, kMagic2)) * sixteenth;
  e[2] = as_half2(and_or(w8, 0x000F000Fu, kMagic2));
  e[3] = as_half2(and_or(w8, 0x00F000F0u, kMagic2)) * sixteenth;
}
// q * scale (q - z exact in fp16) in the activations' type, rounded once
template <bool BF>
__device__ __forceinline__ uint32_t scaled_codes(half2v q, half2v scale) {
  if constexpr (BF)
    return pack_bf16x2(__builtin_fmaf((float)q[0], (float)scale[0], 0.f), __builtin_fmaf((float)q[1], (float)scale[1], 0.f));
  else
    return __builtin_bit_cast(uint32_t, q * scale);
}

// ---- the plan -------------------------------------------------------------------------

struct ExpertTile {
  int expert, row0, rows;  // sorted rows row0 .. row0 + rows - 1
  int first, count;        // the expert's tiles
  int pad[3];
};
struct Plan {
  const int32_t *order;      // [S] slots, sorted by expert (those that name one)
  const ExpertTile *tiles;
  const int32_t *count;      // tiles there are
  // without a plan (order null): the call's ids, at most kSmallSlots of them (small_tile)
  const int32_t *ids;
  int S, E;
};

constexpr int kPlanThreads = 1024;  // and the most experts

// Counts per expert, their prefix sums (and those of their tiles), then each slot to its
// place.  A workgroup places a share of the slots and counts all of them, those before its
// share apart, so none waits for another: placing is what takes long, a store to a
// line of its own for each slot.  32768 slots over 64 experts: 8.4 us, and by
// one workgroup 21.
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const int32_t *ids, int S, int E, int tile_rows,
                                                            int32_t *order, ExpertTile *tiles,
                                                            int32_t *tile_count) {
  __shared__ int before[kPlanThreads], count[kPlanThreads];
  __shared__ int2 part[kPlanThreads / 64];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int share = (S + (int)gridDim.x - 1) / (int)gridDim.x, s0 = share * (int)blockIdx.x, s1 = min(S, s0 + share);
  before[t] = count[t] = 0;
  __syncthreads();
  constexpr int kAhead = 8;  // ids per thread and turn, loaded together
  for (int i0 = t; i0 < S; i0 += kAhead * kPlanThreads) {
    int e[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) e[u] = i0 + u * kPlanThreads < S ? ids[i0 + u * kPlanThreads] : -1;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (e[u] >= 0 && e[u] < E) atomicAdd(i0 + u * kPlanThreads < s0 ? &before[e[u]] : &count[e[u]], 1);
  }
  __syncthreads();
  const int rows = before[t] + count[t], mine = (rows + tile_rows - 1) / tile_rows;
  int a = rows, b = mine;  // inclusive sums over the wave, then over the waves
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int pa = __shfl_up(a, o), pb = __shfl_up(b, o);
    if (lane >= o) {
      a += pa;
      b += pb;
    }
  }
  if (lane == 63) part[wave] = make_int2(a, b);
  __syncthreads();
  for (int w = 0; w < wave; ++w) {
    a += part[w].x;
    b += part[w].y;
  }
  const int first = a - rows;
  if (blockIdx.x == 0) {
    for (int i = 0; i < mine; ++i)
      tiles[b - mine + i] = {t, first + i * tile_rows, min(tile_rows, rows - i * tile_rows), b - mine, mine, {}};
    if (t == kPlanThreads - 1) *tile_count = b;
  }
  before[t] += first;  // where the share's next slot of expert t goes
  __syncthreads();
  for (int i0 = s0 + t; i0 < s1; i0 += kAhead * kPlanThreads) {
    int e[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) e[u] = i0 + u * kPlanThreads < s1 ? ids[i0 + u * kPlanThreads] : -1;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) e[u] = e[u] >= 0 && e[u] < E ? atomicAdd(&before[e[u]], 1) : -1;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (e[u] >= 0) order[e[u]] = i0 + u * kPlanThreads;
  }
}

// ---- operands and epilogues shared by the products -------------------------------------------

enum { kGatedOut = 0, kRowsOut = 1 };

struct ExpertArgs {
  Plan plan;
  const void *A;          // gathered: [tokens][K] rows; else [sorted rows][K]
  const uint8_t *Wq[2];   // expert 0's weights (gated: gate and up)
  const _Float16 *scales[2], *zeros[2];
  size_t code_bytes, meta_count;  // from one expert to the next
  int K, N;               // of one weight: outputs are N wide
  int k, tokens;          // slots per token; tokens of A when gathered
  const float *weights;   // [slots]
  const _Float16 *s_down; // [E][N] or null (gated)
  void *G, *U;            // [slots][N] or null (gated)
  void *H;                // gated: [sorted rows][N]
  float *part;            // rows: [slabs][slots][N], weighted
  int act, columns;       // columns: workgroups along the outputs
  int slabs;              // parts of the contraction (tiles of 32 rows and more)
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void *p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void *)p, (short)0, (int)min((size_t)0x7fffffff, bytes), kRsrcWord3);
}

// The tile and column block of workgroup `block` (false: past the last).  The active
// workgroups are renumbered so that each XCD (they go round the eight) takes one run of them,
// and within an expert the tiles of one column block are neighbours, which share its
// weights in the XCD's L2.
__device__ __forceinline__ bool place(const Plan &plan, int columns, int block, ExpertTile &tile, int &column) {
  const int total = uniform_int(*plan.count) * columns, run = (total + 7) >> 3;
  const int local = (block & 7) * run + (block >> 3);
  if ((block >> 3) >= run || local >= total) return false;
  const ExpertTile &any = plan.tiles[local / columns];  // (of the same expert)
  const int first = uniform_int(any.first), count = uniform_int(any.count), at = local - first * columns;
  column = at / count;
  const ExpertTile &t = plan.tiles[first + at - column * count];
  tile = {uniform_int(t.expert), uniform_int(t.row0), uniform_int(t.rows), first, count, {}};
  return true;
}

// One part of the contraction where it is split: stages begin .. end - 1 of `stages`, and
// `column` without the part.
struct Part {
  int slab, begin, end;
};
__device__ __forceinline__ Part part_of(int &column, int columns, int slabs, int stages) {
  const int slab = column / columns;
  column -= slab * columns;
  return {slab, (int)((long long)stages * slab / slabs), (int)((long long)stages * (slab + 1) / slabs)};
}

// The same without a plan, for at most 16 slots, whose ids are the first lanes of a wave: a
// tile is all of an expert's slots, numbered by the first of them.  `slots` gets the slot of
// each row.  A launch less, for a search in every workgroup: 25.8 us for the call rather than
// 29.2 with a plan at 8 slots (64 experts of 1024 x 4096), 160 and 162 at 16 (8 experts of
// 14336 x 4096), but with the search over 64 slots 89 and 82.
constexpr int kSmallSlots = 16;

__device__ __forceinline__ bool small_tile(const Plan &plan, int columns, int block, ExpertTile &tile, int &column, int *slots) {
  const int lane = threadIdx.x & 63;
  const int e = lane < plan.S ? plan.ids[lane] : -1;
  const bool named = e >= 0 && e < plan.E;
  int rank = 0;  // how many slots before the lane's name its expert
#pragma unroll
  for (int i = 0; i < kSmallSlots - 1; ++i) rank += __builtin_amdgcn_readlane(e, i) == e && i < lane ? 1 : 0;
  uint64_t first = __ballot(named && rank == 0);
  const int total = (int)__builtin_popcountll(first) * columns, run = (total + 7) >> 3;
  const int local = (block & 7) * run + (block >> 3);
  if ((block >> 3) >= run || local >= total) return false;
  const int t = local / columns;
  column = local - t * columns;
  for (int i = 0; i < t; ++i) first &= first - 1;
  const int te = __builtin_amdgcn_readlane(e, __builtin_ctzll(first));
  const bool in = named && e == te;
  tile = {te, 0, (int)__builtin_popcountll(__ballot(in)), 0, 1, {}};
  if (in && threadIdx.x < 64) slots[rank] = lane;
  return true;
}

// A wave's 16 x 64 fp32 sums go through 4 KB of its own LDS on their way out, so that a
// lane has neighbouring columns of one row and stores 16 bytes of them: straight from
// the MFMA's layout, 16 columns of 4 bytes at a time, the down product of 32768 slots of
// 4096 (1024 deep) took 700 us, and 455 us this way.  Column blocks of 16 are swapped by row
// (XOR with row / 4 % 4), so that the four rows that a write touches lie in different banks.
__device__ __forceinline__ int staged(int row, int col) { return row * 64 + (col ^ ((row >> 2 & 3) * 16)); }
__device__ __forceinline__ void stage_block(float *stage, int j, int c, int r, float4v x) {
#pragma unroll
  for (int v = 0; v < 4; ++v) stage[staged(4 * c + v, 16 * j + r)] = x[v];
}
// (the lanes of a wave write, then read: their LDS operations stay in order)
__device__ __forceinline__ void stage_done() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

template <bool BF>
__device__ __forceinline__ u32x4 pack8(const float4v &a, const float4v &b) {
  u32x4 o;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    o[q] = (uint32_t)f32_to_act<BF>(a[2 * q]) | (uint32_t)f32_to_act<BF>(a[2 * q + 1]) << 16;
    o[2 + q] = (uint32_t)f32_to_act<BF>(b[2 * q]) | (uint32_t)f32_to_act<BF>(b[2 * q + 1]) << 16;
  }
  return o;
}

// The wave's 16 x 32 block of 16-bit values (two 16-column blocks of x in fp32) of rows row0 ..
// of the tile, columns n0 ..: each lane 8 columns of one row.  ROW(row) is the row's address.
template <bool BF, typename ROW>
__device__ __forceinline__ void store_16x32(float *stage, int lane, int row0, int rows, const float4v (&x)[2], ROW &&row) {
  const int c = lane >> 4, r = lane & 15;
  stage_block(stage, 0, c, r, x[0]);
  stage_block(stage, 1, c, r, x[1]);
  stage_done();
  const int m = lane >> 2, n = 8 * (lane & 3);
  const float4v a = *reinterpret_cast<const float4v *>(stage + staged(m, n));
  const float4v b = *reinterpret_cast<const float4v *>(stage + staged(m, n + 4));
  stage_done();
  if (row0 + m < rows) *reinterpret_cast<u32x4 *>(row(row0 + m) + n) = pack8<BF>(a, b);
}

// 16 rows of G and U (and H from them), 32 columns from n0: g and u hold two 16-column
// blocks each.  SLOT(row) is a tile's row's slot, HROW(row) its row of H.  H is rounded because it
// is the next product's MFMA operand: Y's error 2.9e-4 rather than 2.1e-4 in fp16, 2.35e-3 rather
// than 1.66e-3 in bf16.
template <bool BF, typename SLOT, typename HROW>
__device__ __forceinline__ void store_gated(const ExpertArgs &P, const ExpertTile &tile, float *stage, int lane, int row0,
                                            int n0, const float4v (&g)[2], const float4v (&u)[2], SLOT &&slot_of,
                                            HROW &&h_row) {
  const int r = lane & 15;
  float4v h[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float sd = P.s_down ? (float)P.s_down[(size_t)tile.expert * P.N + n0 + 16 * j + r] : 1.f;
#pragma unroll
    for (int v = 0; v < 4; ++v) h[j][v] = act_value(g[j][v], P.act) * u[j][v] * sd;
  }
  store_16x32<BF>(stage, lane, row0, tile.rows, h, [&](int m) {
    return static_cast<uint16_t *>(P.H) + (size_t)h_row(m) * P.N + n0;
  });
  if (!P.G) return;
  store_16x32<BF>(stage, lane, row0, tile.rows, g, [&](int m) {
    return static_cast<uint16_t *>(P.G) + (size_t)slot_of(m) * P.N + n0;
  });
  store_16x32<BF>(stage, lane, row0, tile.rows, u, [&](int m) {
    return static_cast<uint16_t *>(P.U) + (size_t)slot_of(m) * P.N + n0;
  });
}

// 16 rows of a slot's contribution, 16 BLOCKS columns from n0, times the slot's weight (or as
// they are: weights null), in fp32.
template <int BLOCKS, typename SLOT>
__device__ __forceinline__ void store_rows(SLOT &&slot_of, const float *weights, float *part, int N, const ExpertTile &tile,
                                           float *stage, int lane, int row0, int n0, const float4v (&y)[BLOCKS]) {
  constexpr int kLanes = 4 * BLOCKS, kRows = 64 / kLanes;  // lanes along a row, rows at a time
#pragma unroll
  for (int j = 0; j < BLOCKS; ++j) stage_block(stage, j, lane >> 4, lane & 15, y[j]);
  stage_done();
  const int n = 4 * (lane % kLanes);
#pragma unroll
  for (int q = 0; q < 16 / kRows; ++q) {
    const int m = kRows * q + lane / kLanes;
    if (row0 + m >= tile.rows) continue;
    const int slot = slot_of(row0 + m);
    float4v x = *reinterpret_cast<const float4v *>(stage + staged(m, n));
    if (weights) x *= weights[slot];
    *reinterpret_cast<float4v *>(part + (size_t)slot * N + n0 + n) = x;
  }
  stage_done();
}

// ---- few rows per expert: streaming -----------------------------------------------------------

// A tile of up to 16 rows, TN 16-row blocks of the weights (gated: alternating gate and
// up), KS waves that each take a KS-th of the contraction and meet in LDS at the end (in
// order).  Bound by HBM: every weight is read once per tile.  Codes and activations
// come straight into registers, DEPTH groups of 128 ahead, with no barrier until the end;
// rows past the tile's are not loaded (their offset lies past the resource).  One token, 2 of 8
// experts of 14336 x 4096 (bf16): gate and up 29.5-30.2 us (4.1-4.2 TB/s), down 15.9-16.2 (3.9).
template <int TN, int KS, int EPI, bool GATHER, bool BF>
__global__ __launch_bounds__(64 * KS) __attribute__((amdgpu_waves_per_eu(TN == 2 ? 4 : 3))) void expert_stream_kernel(ExpertArgs P) {
  constexpr int DEPTH = 2;
  constexpr int STEP = EPI == kGatedOut ? 2 : 1;
  __shared__ float4v red[KS][TN][64];
  __shared__ __attribute__((aligned(16))) float stage[TN / (2 * STEP)][1024];
  __shared__ int slots[16];
  const bool small = P.plan.order == nullptr;
  ExpertTile tile;
  int column;
  if (small) {
    if (!small_tile(P.plan, P.columns, blockIdx.x, tile, column, slots)) return;
  } else {
    if (!place(P.plan, P.columns, blockIdx.x, tile, column)) return;
    if ((int)threadIdx.x < tile.rows) slots[threadIdx.x] = P.plan.order[tile.row0 + threadIdx.x];
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = uniform_int(threadIdx.x >> 6), c = lane >> 4, r = lane & 15;
  const int K = P.K, N = P.N, G = K / kGroup, NB = N / kTileRows;
  const int vb0 = column * TN;  // first row block (gated: of the alternating ones)

  // rows of A: gathered, of the tokens; else of H, which has the tile's rows in a run, or (without
  // a plan) every slot's row
  const __amdgpu_buffer_rsrc_t ars =
      GATHER ? resource(P.A, (size_t)P.tokens * K * 2)
             : small ? resource(P.A, (size_t)P.plan.S * K * 2)
                     : resource(static_cast<const uint16_t *>(P.A) + (size_t)tile.row0 * K, (size_t)tile.rows * K * 2);
  int aoff = kOutOfRange;
  if (r < tile.rows) aoff = ((GATHER ? slots[r] / P.k : small ? slots[r] : r) * K + 8 * c) * 2;
  __amdgpu_buffer_rsrc_t wrs[STEP], srs[STEP], zrs[STEP];
  const size_t code0 = tile.expert * P.code_bytes, meta0 = tile.expert * P.meta_count;
#pragma unroll
  for (int i = 0; i < STEP; ++i) {
    wrs[i] = resource(P.Wq[i] + code0, P.code_bytes);
    srs[i] = resource(P.scales[i] + meta0, P.meta_count * 2);
    zrs[i] = resource(P.zeros[i] + meta0, P.meta_count * 2);
  }
  const int tile_stride = NB * kTileBytes, meta_stride = NB * kTileRows * kMetaQuad * 2;
  const int g0 = G * wave / KS, g1 = G * (wave + 1) / KS;

  struct Stage {
    u32x4 a[4], code[TN];
    uint32_t sc[TN], zp[TN];
  } st[DEPTH];
  auto load = [&](int g, Stage &s) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int rb = min(vb0 + j, STEP * NB - 1) / STEP;  // (blocks past N: the last again, not stored)
      s.code[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                wrs[j % STEP], lane * 16, g * tile_stride + rb * kTileBytes, 0));
      const int qo = (g / kMetaQuad) * meta_stride + (rb * kTileRows * kMetaQuad + g % kMetaQuad) * 2;
      s.sc[j] = __builtin_amdgcn_raw_buffer_load_b16(srs[j % STEP], r * kMetaQuad * 2, qo, 0);
      s.zp[j] = __builtin_amdgcn_raw_buffer_load_b16(zrs[j % STEP], r * kMetaQuad * 2, qo, 0);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
      s.a[t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ars, aoff, g * kGroup * 2 + 64 * t, 0));
  };
  float4v acc[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) acc[j] = float4v{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Stage &s) {
    float4v xs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 4; ++t) xs = mfma<BF>(s.a[t], ones_operand<BF>(), xs);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      float4v p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < 4; ++t) p = mfma<BF>(s.a[t], code_operand<BF>(s.code[j][t]), p);
      const float sc = (float)__builtin_bit_cast(_Float16, (uint16_t)s.sc[j]);
      const float z = kCodeBase<BF> + (float)__builtin_bit_cast(_Float16, (uint16_t)s.zp[j]);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[j][v] = __builtin_fmaf(sc, __builtin_fmaf(-z, xs[v], p[v]), acc[j][v]);
    }
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (g0 + d < g1) load(g0 + d, st[d]);
  for (int g = g0; g < g1; g += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (g + d >= g1) break;
      compute(st[d]);
      if (g + d + DEPTH < g1) load(g + d + DEPTH, st[d]);
    }
  }

#pragma unroll
  for (int j = 0; j < TN; ++j) red[wave][j][lane] = acc[j];
  __syncthreads();
  // waves 0 .. finish 32 columns each (gated: of H, from 64 sums)
  constexpr int OUT = 2 * STEP;
  if (wave >= TN / OUT) return;
  float4v y[OUT];
#pragma unroll
  for (int i = 0; i < OUT; ++i) {
    y[i] = red[0][OUT * wave + i][lane];
#pragma unroll
    for (int w = 1; w < KS; ++w) y[i] += red[w][OUT * wave + i][lane];
  }
  const int n0 = (vb0 + OUT * wave) / STEP * kTileRows;
  if (n0 >= N) return;  // (N is a multiple of 128: all 32 columns are there)
  auto slot_of = [&](int m) { return slots[m]; };
  if constexpr (EPI == kGatedOut)
    store_gated<BF>(P, tile, stage[wave], lane, 0, n0, {y[0], y[2]}, {y[1], y[3]}, slot_of,
                    [&](int m) { return small ? slots[m] : tile.row0 + m; });
  else
    store_rows<2>(slot_of, P.weights, P.part, N, tile, stage[wave], lane, 0, n0, {y[0], y[1]});
}

// ---- many rows per expert: LDS tiles -----------------------------------------------------------

// A tile of 16 TM rows and 256 outputs (gated: 128 of G and of U), four waves of 16 TM x
// 64, a group of 128 of the contraction per stage: the rows go into LDS with DMA loads
// (double-buffered, XOR-swizzled 16-byte chunks, one barrier a stage), the wave's code
// tiles into registers one stage ahead.
//
// The codes are multiplied as they are (code_operand) and the group's scale and zero
// point applied to its fp32 sums, so no weight is rounded and the decoding costs 7
// instructions per 8 weights; it is the sums that cost two FMAs per element and group,
// half of what their four MFMAs take.  The sums of a group's activations, which the zero
// points multiply, are MFMAs with ones: wave i takes those of row block i, and they reach
// the other waves through LDS a stage later.  64 tokens, 8 of 64 experts of 1024 x 4096 (fp16, 32
// rows): gate and up 58-60 us (4.7-4.9 TB/s of weights), down 37-38.5 (3.7-3.8, and 8 MB written); 48 rows
// per expert and more are bound by the issue of vector instructions (4.35 to an MFMA).
template <int TM, int EPI, bool GATHER, bool BF>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void expert_tile_kernel(ExpertArgs P) {
  constexpr int TN = 4, BM = 16 * TM, STEP = EPI == kGatedOut ? 2 : 1;
  constexpr int kRowChunks = kGroup / 8, kDma = BM * kRowChunks / 256;  // DMA loads per wave and stage (TM)
  // (an array for each buffer: from one array the compiler cannot tell the buffer that is
  // read from the one that a DMA load in flight writes, and waits for the load)
  __shared__ __attribute__((aligned(16))) _Float16 As0[BM * kGroup], As1[BM * kGroup];
  __shared__ float4v Xs0[BM / 4], Xs1[BM / 4];
  __shared__ __attribute__((aligned(16))) float stage[4][1024];
  ExpertTile tile;
  int column;
  if (!place(P.plan, P.columns * P.slabs, blockIdx.x, tile, column)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform_int(tid >> 6), c = lane >> 4, r = lane & 15;
  const int K = P.K, N = P.N, NB = N / kTileRows;
  const Part part = part_of(column, P.columns, P.slabs, K / kGroup);
  const int G0 = part.begin, G = part.end - G0;  // the part's first group, and how many

  // wave load u fills LDS chunks p = (u * 4 + wave) * 64 + lane: row p / 16 = 16 u + 4 wave +
  // lane / 16, physical chunk p % 16, holding logical chunk lc = (p % 16) ^ (row % 16), the same
  // for every u.  Rows past the tile's lie past the resource and read zeros.
  const __amdgpu_buffer_rsrc_t ars =
      GATHER ? resource(P.A, (size_t)P.tokens * K * 2)
             : resource(static_cast<const uint16_t *>(P.A) + (size_t)tile.row0 * K, (size_t)tile.rows * K * 2);
  const int arow = 4 * wave + c, lc = r ^ arow;
  int aoff[GATHER ? kDma : 1];
  aoff[0] = (arow * K + 8 * lc) * 2;
  if constexpr (GATHER) {
#pragma unroll
    for (int u = 0; u < kDma; ++u) {
      aoff[u] = kOutOfRange;
      if (16 * u + arow < tile.rows)
        aoff[u] = (P.plan.order[tile.row0 + 16 * u + arow] / P.k * K + 8 * lc) * 2;
    }
  }
  auto load_a = [&](int g, int buf) {
#pragma unroll
    for (int u = 0; u < kDma; ++u) {
      const int vo = GATHER ? aoff[GATHER ? u : 0] : aoff[0] + 32 * u * K;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          ars, (__attribute__((address_space(3))) void *)((buf ? As1 : As0) + (u * 4 + wave) * 64 * 8), 16, vo,
          (G0 + g) * kGroup * 2, 0, 0);
    }
  };
  __amdgpu_buffer_rsrc_t wrs[STEP], srs[STEP], zrs[STEP];
  const size_t code0 = tile.expert * P.code_bytes, meta0 = tile.expert * P.meta_count;
#pragma unroll
  for (int i = 0; i < STEP; ++i) {
    wrs[i] = resource(P.Wq[i] + code0, P.code_bytes);
    srs[i] = resource(P.scales[i] + meta0, P.meta_count * 2);
    zrs[i] = resource(P.zeros[i] + meta0, P.meta_count * 2);
  }
  const int vb0 = (column * 4 + wave) * TN;
  const int tile_stride = NB * kTileBytes, meta_stride = NB * kTileRows * kMetaQuad * 2;
  struct Codes {
    u32x4 w[TN];
  };
  uint32_t sc[TN], zp[TN];  // raw fp16 scale and zero point of the latest group
  // (32 rows: an expert has a tile or two, and streaming loads leave the L2 to the rest: gate and up
  // of 64 experts as above 60 -> 58 us, down 38.5 -> 36.6; weights that all fit in the caches and
  // are there already, 76 MB, 40 -> 42)
  constexpr int kStreaming = TM == 2 ? 2 : 0;
  auto load_codes = [&](int g, Codes &b) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int rb = min(vb0 + j, STEP * NB - 1) / STEP;
      b.w[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             wrs[j % STEP], lane * 16, (G0 + g) * tile_stride + rb * kTileBytes, kStreaming));
    }
  };
  auto load_meta = [&](int step) {
    const int g = G0 + step;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int rb = min(vb0 + j, STEP * NB - 1) / STEP;
      const int qo = (g / kMetaQuad) * meta_stride + (rb * kTileRows * kMetaQuad + g % kMetaQuad) * 2;
      sc[j] = __builtin_amdgcn_raw_buffer_load_b16(srs[j % STEP], r * kMetaQuad * 2, qo, 0);
      zp[j] = __builtin_amdgcn_raw_buffer_load_b16(zrs[j % STEP], r * kMetaQuad * 2, qo, 0);
    }
  };

  constexpr int kTiles = TM * TN;
  float4v acc[kTiles], p[kTiles];  // 16 x 16 block TN i + j: the sum, and the latest group's product
#pragma unroll
  for (int t = 0; t < kTiles; ++t) acc[t] = p[t] = float4v{0.f, 0.f, 0.f, 0.f};
  u32x4 bop[2][TN];  // operands of this k step and the next
  float scale[TN], zs[TN];  // of the group before: scale, scale * (base + zero point)
  auto take_meta = [&]() {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      scale[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)sc[j]);
      zs[j] = scale[j] * (kCodeBase<BF> + (float)__builtin_bit_cast(_Float16, (uint16_t)zp[j]));
    }
  };
  // element n (of 4 kTiles) of the zero points' share, row blocks in order
  auto take_zero = [&](int n, const float4v &xs) {
    const int i = n / (4 * TN), j = n / 4 % TN, v = n % 4;
    acc[TN * i + j][v] = __builtin_fmaf(-zs[j], xs[v], acc[TN * i + j][v]);
  };

  // One group per step: wait until this group's loads (issued a step ago) and the row sums
  // of the group before are in LDS and every wave is past the previous step, issue the next
  // group's loads, multiply.  Past the range they re-read the last group.
  //
  // An MFMA runs for 16 cycles and takes 4 to issue; only vector instructions that stand right
  // behind it run meanwhile (16 MFMAs and 48 FMAs take 141 ns in turn by threes, 124 ns without the
  // FMAs, and 226 ns one after the other, with one to four waves on the SIMD).  So each MFMA
  // comes with its share of the rest, held in place by scheduling barriers: in the first k
  // step the block's sum takes the product of the group before (4 FMAs), just before that
  // product's registers are written again; in the others, the zero points' share of that
  // group (2, 1 and 1 FMAs); in all, part of the next k step's operands (7 instructions for 4).
  auto step = [&](int g, Codes &cur, Codes &nxt, int buf) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    take_meta();
    const int gn = min(g + 1, G - 1);
    load_codes(gn, nxt);
    load_a(gn, buf ^ 1);
    // (LDS addresses are formed again in every step: kept, they would take the registers
    // that the operands need)
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int sc_ = ln >> 4, sr = ln & 15, first = (sr * kGroup + 8 * (sc_ ^ sr)) * 2;
    const char *as = reinterpret_cast<const char *>(buf ? As1 : As0);
    auto read_a = [&](int n) {  // k step n / TM, row block n % TM: chunk (4 tt + c) ^ r of row r
      return *reinterpret_cast<const u32x4 *>(as + ((first ^ (64 * (n / TM))) + 32 * kGroup * (n % TM)));
    };
    u32x4 a[3], own;  // two row blocks ahead; the row block whose sums this wave takes
    a[0] = read_a(0);
    a[1] = read_a(1);
    float4v xs_prev, xs_next, xs = {0.f, 0.f, 0.f, 0.f};
    auto xs_of = [&](int i, int b) { return (b ? Xs1 : Xs0)[4 * i + sc_]; };
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const int i = t / TN, j = t % TN, n = TM * tt + i;
        if (tt == 0) {
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[t][v] = __builtin_fmaf(scale[j], p[t][v], acc[t][v]);
        }
        if (j == 0 && n + 2 < 4 * TM) a[(n + 2) % 3] = read_a(n + 2);
        if (t == kTiles / 2)
          own = *reinterpret_cast<const u32x4 *>(as + ((first ^ (64 * tt)) + 32 * kGroup * (wave % TM)));
        if (tt == 1 && t == 0) load_meta(g);
        if (tt == 0 && t == kTiles - TN) xs_prev = xs_of(0, buf ^ 1);
        p[t] = mfma<BF>(a[n % 3], bop[tt & 1][j], tt ? p[t] : float4v{0.f, 0.f, 0.f, 0.f});
        // the next k step's operands, 16 words of them over the step's MFMAs
#pragma unroll
        for (int q = 0; q < 16 / kTiles; ++q) {
          const int m = t * (16 / kTiles) + q;
          bop[(tt + 1) & 1][m / 4][m % 4] =
              code_part<BF>(tt < 3 ? cur.w[m / 4][tt < 3 ? tt + 1 : 0] : nxt.w[m / 4][0], m % 4);
        }
        // the zero points' share: half of it, then a quarter each
        if (tt > 0) {
          constexpr int kPer = 4 * TN;
          const int n0 = tt == 1 ? 2 * t : kTiles * tt + t, nn = tt == 1 ? 2 : 1;
#pragma unroll
          for (int q = 0; q < nn; ++q) {
            const int e = n0 + q;
            if (e % kPer == 0 && e > 0) xs_prev = xs_next;
            if (e % kPer == kPer / 2 && e / kPer + 1 < TM) xs_next = xs_of(e / kPer + 1, buf ^ 1);
            take_zero(e, xs_prev);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      xs = mfma<BF>(own, ones_operand<BF>(), xs);
    }
    (buf ? Xs1 : Xs0)[4 * (wave % TM) + sc_] = xs;  // (the same from all 16 lanes of a row, and every TM-th wave)
  };
  Codes c0, c1;
#pragma unroll
  for (int j = 0; j < TN; ++j) sc[j] = zp[j] = 0;
  if (tid < BM / 4) Xs1[tid] = float4v{0.f, 0.f, 0.f, 0.f};  // (before the first group: 0 times 0)
  load_codes(0, c0);
  load_a(0, 0);
#pragma unroll
  for (int m = 0; m < 16; ++m) bop[0][m / 4][m % 4] = code_part<BF>(c0.w[m / 4][0], m % 4);
  // (no branch between the two steps, or what the second alone uses is moved out of the first)
  int g = 0;
  for (; g + 1 < G; g += 2) {
    step(g, c0, c1, 0);
    step(g + 1, c1, c0, 1);
  }
  if (g < G) step(g, c0, c1, 0);
  // (the last step's DMA must land before the workgroup's LDS is released)
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  take_meta();
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const float4v xs = ((G - 1) & 1 ? Xs1 : Xs0)[4 * i + c];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        acc[TN * i + j][v] = __builtin_fmaf(scale[j], p[TN * i + j][v], acc[TN * i + j][v]);
        take_zero(4 * (TN * i + j) + v, xs);
      }
  }

  // (the lane's place again, rather than in registers through the loop)
  const int at = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  const int n0 = vb0 / STEP * kTileRows;
  if (n0 >= N) return;  // (N is a multiple of 128: a wave's columns are all there or none)
  auto slot_of = [&](int m) { return P.plan.order[tile.row0 + m]; };
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    if (16 * i >= tile.rows) break;
    if constexpr (EPI == kGatedOut)
      store_gated<BF>(P, tile, stage[wave], at, 16 * i, n0, {acc[TN * i], acc[TN * i + 2]},
                      {acc[TN * i + 1], acc[TN * i + 3]}, slot_of, [&](int m) { return tile.row0 + m; });
    else
      store_rows<4>(slot_of, P.weights, P.part + (size_t)part.slab * P.plan.S * N, N, tile, stage[wave], at, 16 * i, n0,
                    {acc[TN * i], acc[TN * i + 1], acc[TN * i + 2], acc[TN * i + 3]});
  }
}

// ---- many more rows: weights rounded once -------------------------------------------------------

// A tile of 128 rows and 256 outputs, laid out as above with twice the rows.  Their sums
// alone take half the registers, which leaves no room for a group's product beside
// them: each weight is rounded to the activations' type, as in the dense layers, and the
// MFMAs add to the sums at once.  Decoding a weight costs three times as much that way,
// shared by twice the rows, and no FMAs follow the MFMAs.  4096 tokens, 8 of 64 experts of
// 1024 x 4096 (bf16): gate and up 598-609 us (550 GFLOP), down 411-423 (275 GFLOP, 537 MB written); by
// 64 rows with exact codes 663 and 453.  MFMAs and vector instructions take turns (41% and 31%
// of the time).  What the rounding costs (16 experts of 2560 x 3584, error of Y against 64 bits in
// the 2-norm): 4.2e-4 in fp16 and 3.7e-3 in bf16, with exact codes 2.9e-4 and 2.35e-3; rounding Y
// alone is 2.1e-4 and 1.66e-3.
template <int EPI, bool GATHER, bool BF>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void expert_wide_kernel(ExpertArgs P) {
  constexpr int TM = 8, TN = 4, BM = 16 * TM, STEP = EPI == kGatedOut ? 2 : 1;
  __shared__ __attribute__((aligned(16))) _Float16 As0[BM * kGroup], As1[BM * kGroup];
  ExpertTile tile;
  int column;
  if (!place(P.plan, P.columns * P.slabs, blockIdx.x, tile, column)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform_int(tid >> 6), c = lane >> 4, r = lane & 15;
  const int K = P.K, N = P.N, NB = N / kTileRows;
  const Part part = part_of(column, P.columns, P.slabs, K / kGroup);

  // rows of A: as in expert_tile_kernel
  const __amdgpu_buffer_rsrc_t ars =
      GATHER ? resource(P.A, (size_t)P.tokens * K * 2)
             : resource(static_cast<const uint16_t *>(P.A) + (size_t)tile.row0 * K, (size_t)tile.rows * K * 2);
  const int arow = 4 * wave + c, lc = r ^ arow;
  int aoff[GATHER ? TM : 1];
  aoff[0] = (arow * K + 8 * lc) * 2;
  if constexpr (GATHER) {
#pragma unroll
    for (int u = 0; u < TM; ++u) {
      aoff[u] = kOutOfRange;
      if (16 * u + arow < tile.rows)
        aoff[u] = (P.plan.order[tile.row0 + 16 * u + arow] / P.k * K + 8 * lc) * 2;
    }
  }
  auto load_a = [&](int g, int buf) {
#pragma unroll
    for (int u = 0; u < TM; ++u) {
      const int vo = GATHER ? aoff[GATHER ? u : 0] : aoff[0] + 32 * u * K;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          ars, (__attribute__((address_space(3))) void *)((buf ? As1 : As0) + (u * 4 + wave) * 64 * 8), 16, vo,
          g * kGroup * 2, 0, 0);
    }
  };
  __amdgpu_buffer_rsrc_t wrs[STEP], srs[STEP], zrs[STEP];
  const size_t code0 = tile.expert * P.code_bytes, meta0 = tile.expert * P.meta_count;
#pragma unroll
  for (int i = 0; i < STEP; ++i) {
    wrs[i] = resource(P.Wq[i] + code0, P.code_bytes);
    srs[i] = resource(P.scales[i] + meta0, P.meta_count * 2);
    zrs[i] = resource(P.zeros[i] + meta0, P.meta_count * 2);
  }
  const int vb0 = (column * 4 + wave) * TN;
  const int tile_stride = NB * kTileBytes, meta_stride = NB * kTileRows * kMetaQuad * 2;
  struct BStage {
    u32x4 code[TN];
    uint32_t sc[TN], zp[TN];  // raw fp16 scale and zero point
  };
  auto load_b = [&](int g, BStage &b) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {  // (blocks past N: the last again, not stored)
      const int rb = min(vb0 + j, STEP * NB - 1) / STEP;
      const int qo = (g / kMetaQuad) * meta_stride + (rb * kTileRows * kMetaQuad + g % kMetaQuad) * 2;
      b.code[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                wrs[j % STEP], lane * 16, g * tile_stride + rb * kTileBytes, 0));
      b.sc[j] = __builtin_amdgcn_raw_buffer_load_b16(srs[j % STEP], r * kMetaQuad * 2, qo, 0);
      b.zp[j] = __builtin_amdgcn_raw_buffer_load_b16(zrs[j % STEP], r * kMetaQuad * 2, qo, 0);
    }
  };

  float4v acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = float4v{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](const BStage &b, int buf) {
    const _Float16 *as = (buf ? As1 : As0) + r * kGroup;
    half2v lo[TN], hi[TN], scale[TN];  // 1024 + z and 64 + z, twice each
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const _Float16 z = __builtin_bit_cast(_Float16, (uint16_t)b.zp[j]), s = __builtin_bit_cast(_Float16, (uint16_t)b.sc[j]);
      const _Float16 zl = (_Float16)1024.f + z, zh = (_Float16)64.f + z;
      lo[j] = half2v{zl, zl};
      hi[j] = half2v{zh, zh};
      scale[j] = half2v{s, s};
    }
    auto dequant = [&](int j, int tt) -> u32x4 {
      half2v e[4];
      code_halves(b.code[j][tt], e);
      return (u32x4){scaled_codes<BF>(e[0] - lo[j], scale[j]), scaled_codes<BF>(e[1] - hi[j], scale[j]),
                     scaled_codes<BF>(e[2] - lo[j], scale[j]), scaled_codes<BF>(e[3] - hi[j], scale[j])};
    };
    // k step tt + 1's weights are dequantized while k step tt's MFMAs run
    u32x4 bop[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) bop[j] = dequant(j, 0);
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      u32x4 bnx[TN];
      if (tt < 3) {
#pragma unroll
        for (int j = 0; j < TN; ++j) bnx[j] = dequant(j, tt + 1);
      }
      const int pc = (4 * tt + c) ^ r;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const u32x4 a = *reinterpret_cast<const u32x4 *>(as + 16 * i * kGroup + 8 * pc);
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mfma<BF>(a, bop[j], acc[i][j]);
      }
      if (tt < 3) {
#pragma unroll
        for (int j = 0; j < TN; ++j) bop[j] = bnx[j];
      }
    }
  };
  BStage b0, b1;
  auto step = [&](int g, BStage &cur, BStage &nxt, int buf) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const int gn = min(g + 1, part.end - 1);  // (past the range: the last again, into what nobody reads)
    load_a(gn, buf ^ 1);
    load_b(gn, nxt);
    compute(cur, buf);
  };
  load_a(part.begin, 0);
  load_b(part.begin, b0);
  for (int g = part.begin; g < part.end; g += 2) {
    step(g, b0, b1, 0);
    if (g + 1 < part.end) step(g + 1, b1, b0, 1);
  }
  // the last step's DMA must land, and every wave be past its reads, before the rows' LDS is
  // used for the outputs
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  const int n0 = vb0 / STEP * kTileRows;
  if (n0 >= N) return;  // (N is a multiple of 128: a wave's columns are all there or none)
  const int at = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  float *stage = reinterpret_cast<float *>(As0) + wave * 1024;
  auto slot_of = [&](int m) { return P.plan.order[tile.row0 + m]; };
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    if (16 * i >= tile.rows) break;
    if constexpr (EPI == kGatedOut)
      store_gated<BF>(P, tile, stage, at, 16 * i, n0, {acc[i][0], acc[i][2]}, {acc[i][1], acc[i][3]}, slot_of,
                      [&](int m) { return tile.row0 + m; });
    else
      store_rows<4>(slot_of, P.weights, P.part + (size_t)part.slab * P.plan.S * N, N, tile, stage, at, 16 * i, n0, acc[i]);
  }
}

// ---- backward products -------------------------------------------------------------------------

enum { kActGradOut = 0, kGradRowsOut = 1 };

struct ExpertGradArgs {
  Plan plan;
  const void *A[2];              // gathered: [tokens][R] rows of dY; else [sorted rows][R]
  const uint8_t *Wt[2], *meta[2];  // expert 0's transposed weights
  size_t code_bytes, meta_bytes; // from one expert to the next
  int R, C;                      // contraction per term, outputs
  int k, tokens;
  const float *weights;          // [slots]
  const _Float16 *s_down;        // [E][C] or null
  const void *G, *U;             // [slots][C]
  void *dG, *dU;                 // [sorted rows][C]
  float *dw_part;                // [slots][4 columns]
  float *part;                   // rows: [slabs][slots][C]
  int act, columns, slabs;
};

// A tile of 16 TM rows and 256 outputs of the sum over the terms of A . D, D [R][C] the
// experts' (q - z) * scale: four waves of 16 TM x 64, 128 rows of one term's D per
// stage.  Rows of A and the stage's scales and zero points (1 KB for 256 outputs) go into LDS
// with DMA loads, the wave's code tiles into registers, all one stage ahead.  The scale
// varies along the contraction here, so it cannot multiply the sums: each weight is
// rounded once to the activations' type, which the MFMA takes, as in the dense layers'
// backward; dG and dU are rounded because they are MFMA operands too.  Both together take the error of dX
// from 2.1e-4 to 3.8e-4 (fp16) and from 1.66e-3 to 3.3e-3 (bf16; 16 experts of 2560 x 3584).
// 2048 tokens, 2 of 8 experts of 14336 x 4096 (bf16): dG and dU 590-605 us (481
// GFLOP), rows 1000-1017 (962 GFLOP).  (Scheduling barriers that pin the loads before the
// MFMAs made the bf16 instances of 128 rows spill: 938 and 861 us on equal work without.)
template <int TM, int EPI, bool GATHER, bool BF>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void expert_grad_kernel(ExpertGradArgs P) {
  constexpr int TN = 4, BM = 16 * TM, TERMS = EPI == kActGradOut ? 1 : 2;
  __shared__ __attribute__((aligned(16))) _Float16 As0[BM * kGroup], As1[BM * kGroup];
  __shared__ __attribute__((aligned(16))) unsigned char Ms0[1024], Ms1[1024];
  __shared__ __attribute__((aligned(16))) float Cs[TM >= 4 ? 1 : 4][TM >= 4 ? 4 : 1024];  // (else in As0)
  ExpertTile tile;
  int column;
  if (!place(P.plan, P.columns * P.slabs, blockIdx.x, tile, column)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform_int(tid >> 6), c = lane >> 4, r = lane & 15;
  const int R = P.R, C = P.C, KB = C / kTileRows, CG = C / kGroup, NG = R / kGroup;
  const Part part = part_of(column, P.columns, P.slabs, TERMS * NG);

  __amdgpu_buffer_rsrc_t ars[TERMS], wrs[TERMS], mrs[TERMS];
#pragma unroll
  for (int i = 0; i < TERMS; ++i) {
    ars[i] = GATHER ? resource(P.A[i], (size_t)P.tokens * R * 2)
                    : resource(static_cast<const uint16_t *>(P.A[i]) + (size_t)tile.row0 * R, (size_t)tile.rows * R * 2);
    wrs[i] = resource(P.Wt[i] + tile.expert * P.code_bytes, P.code_bytes);
    mrs[i] = resource(P.meta[i] + tile.expert * P.meta_bytes, P.meta_bytes);
  }
  // rows of A: as in expert_tile_kernel
  const int arow = 4 * wave + c, lc = r ^ arow;
  int aoff[GATHER ? TM : 1];
  aoff[0] = (arow * R + 8 * lc) * 2;
  if constexpr (GATHER) {
#pragma unroll
    for (int u = 0; u < TM; ++u) {
      aoff[u] = kOutOfRange;
      if (16 * u + arow < tile.rows)
        aoff[u] = (P.plan.order[tile.row0 + 16 * u + arow] / P.k * R + 8 * lc) * 2;
    }
  }
  auto load_a = [&](int stage, int buf) {
    const int ti = TERMS > 1 && stage >= NG ? 1 : 0, g = stage - ti * NG;
    // (an array element passed straight to the builtin keeps the kernel from being
    // instantiated in the host compilation)
    const __amdgpu_buffer_rsrc_t rs = ti ? ars[TERMS - 1] : ars[0], ms = ti ? mrs[TERMS - 1] : mrs[0];
#pragma unroll
    for (int u = 0; u < TM; ++u) {
      const int vo = GATHER ? aoff[GATHER ? u : 0] : aoff[0] + 32 * u * R;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void *)((buf ? As1 : As0) + (u * 4 + wave) * 64 * 8), 16, vo,
          g * kGroup * 2, 0, 0);
    }
    // scales and zero points of the block's two quantization groups (or its one, twice): 256 bytes a wave
    const int mo = ((column * 2 + 1 < CG ? wave : wave & 1) * 64 + lane) * 4;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        ms, (__attribute__((address_space(3))) void *)((buf ? Ms1 : Ms0) + wave * 256), 4, mo,
        (g * CG + column * 2) * kMetaBytes, 0, 0);
  };
  const int kb0 = (column * 4 + wave) * TN, tile_stride = KB * kTileBytes;
  struct BStage {
    u32x4 code[TN];
  };
  auto load_b = [&](int stage, BStage &b) {
    const int ti = TERMS > 1 && stage >= NG ? 1 : 0, g = stage - ti * NG;
    const __amdgpu_buffer_rsrc_t rs = ti ? wrs[TERMS - 1] : wrs[0];
#pragma unroll
    for (int j = 0; j < TN; ++j)  // (column blocks past C: the last again, not stored)
      b.code[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                rs, lane * 16,
                                                g * tile_stride + min(kb0 + j, KB - 1) * kTileBytes, 0));
  };
  const int ul = wave >> 1;  // the wave's quantization group among the block's two

  float4v acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = float4v{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](const BStage &b, int buf) {
    const _Float16 *as = (buf ? As1 : As0) + r * kGroup;
    const _Float16 *ms = reinterpret_cast<const _Float16 *>((buf ? Ms1 : Ms0) + ul * kMetaBytes) + 8 * c;
    struct Meta {
      half8 scale, bias;
    };
    auto meta_at = [&](int tt) -> Meta {
      return {*reinterpret_cast<const half8 *>(ms + 32 * tt), *reinterpret_cast<const half8 *>(ms + kGroup + 32 * tt)};
    };
    auto dequant = [&](int j, int tt, const Meta &m) -> u32x4 {
      half2v e[4];
      code_halves(b.code[j][tt], e);
      u32x4 out;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const half2v bias = {m.bias[2 * p], m.bias[2 * p + 1]}, scale = {m.scale[2 * p], m.scale[2 * p + 1]};
        out[p] = scaled_codes<BF>(e[p] - bias, scale);
      }
      return out;
    };
    // k step tt + 1's weights are dequantized while k step tt's MFMAs run
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
      const int pc = (4 * tt + c) ^ r;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const u32x4 a = *reinterpret_cast<const u32x4 *>(as + 16 * i * kGroup + 8 * pc);
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mfma<BF>(a, bop[j], acc[i][j]);
      }
      if (tt < 3) {
#pragma unroll
        for (int j = 0; j < TN; ++j) bop[j] = bnx[j];
      }
    }
  };
  BStage b0, b1;
  auto step = [&](int i, BStage &cur, BStage &nxt, int buf) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const int next = min(i + 1, part.end - 1);  // (past the range: the last again, into what nobody reads)
    load_a(next, buf ^ 1);
    load_b(next, nxt);
    compute(cur, buf);
  };
  load_a(part.begin, 0);
  load_b(part.begin, b0);
  for (int i = part.begin; i < part.end; i += 2) {
    step(i, b0, b1, 0);
    if (i + 1 < part.end) step(i + 1, b1, b0, 1);
  }
  // the last step's DMA must land, and every wave be past its reads, before the rows' LDS is
  // used for the outputs
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  if (kb0 >= KB) return;  // (C is a multiple of 128: a wave's 64 outputs are all there or none)
  const int at = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  float *stage = TM >= 4 ? reinterpret_cast<float *>(As0) + wave * 1024 : Cs[TM >= 4 ? 0 : wave];
  const int n0 = kb0 * kTileRows;
  if constexpr (EPI == kGradRowsOut) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
      if (16 * i < tile.rows) store_rows<4>([&](int m) { return P.plan.order[tile.row0 + m]; }, nullptr,
                      P.part + (size_t)part.slab * P.plan.S * C, C, tile, stage, at, 16 * i, n0, acc[i]);
  } else {
    // (a loop, with one copy of the activations' code: only the sums are picked by number)
#pragma unroll 1
    for (int i = 0; 16 * i < tile.rows; ++i) {
#pragma unroll
      for (int k = 0; k < TM; ++k) {
        if (k != i) continue;
#pragma unroll
        for (int j = 0; j < TN; ++j) stage_block(stage, j, at >> 4, at & 15, acc[k][j]);
      }
      stage_done();
      const int n = 8 * (at & 7);  // eight columns per lane, eight rows at a time
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int m = 8 * q + (at >> 3), row = 16 * i + m;
        const bool in = row < tile.rows;
        const size_t sorted = (size_t)(tile.row0 + (in ? row : 0));
        const int slot = P.plan.order[sorted];
        const float w = P.weights[slot];
        const size_t from = (size_t)slot * C + n0 + n;
        const u32x4 g8 = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(P.G) + from);
        const u32x4 u8 = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(P.U) + from);
        half8 sd;
        if (P.s_down) sd = load_half8(P.s_down + (size_t)tile.expert * C + n0 + n);
        float4v dg[2], du[2];
        float dw = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4v x = *reinterpret_cast<const float4v *>(stage + staged(m, n + 4 * h));
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int k = 4 * h + v;
            const float g = act_to_f32<BF>((uint16_t)(g8[k / 2] >> (16 * (k & 1))));
            const float u = act_to_f32<BF>((uint16_t)(u8[k / 2] >> (16 * (k & 1))));
            const float dh = P.s_down ? x[v] * (float)sd[k] : x[v], a = act_value(g, P.act);
            dw = __builtin_fmaf(dh, a * u, dw);
            dg[h][v] = w * dh * u * act_grad(g, P.act);
            du[h][v] = w * dh * a;
          }
        }
#pragma unroll
        for (int o = 1; o < 8; o *= 2) dw += __shfl_xor(dw, o);
        if (in) {
          const size_t to = sorted * C + n0 + n;
          *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(P.dG) + to) = pack8<BF>(dg[0], dg[1]);
          *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(P.dU) + to) = pack8<BF>(du[0], du[1]);
          if ((at & 7) == 0) P.dw_part[(size_t)slot * (4 * P.columns) + column * 4 + wave] = dw;
        }
      }
      stage_done();
    }
  }
}

// dw of each slot: its partial sums over the first `parts` of `stride`, one wave per slot, in a
// fixed order; 0 for a slot that names no expert.
template <bool BF>
__global__ __launch_bounds__(256) void weight_grad_kernel(const int32_t *ids, const float *part, int stride, int parts,
                                                          int S, int E, void *dw, bool f32) {
  const int slot = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (slot >= S) return;
  const int e = ids[slot];
  float s = 0.f;
  if (e >= 0 && e < E)
    for (int i = lane; i < parts; i += 64) s += part[(size_t)slot * stride + i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if (lane != 0) return;
  if (f32)
    static_cast<float *>(dw)[slot] = s;
  else
    static_cast<uint16_t *>(dw)[slot] = f32_to_act<BF>(s);
}

// ---- joining a token's slots ---------------------------------------------------------------------

struct CombineArgs {
  const int32_t *ids;
  const float *part;         // [slabs][slots][D]
  const void *add;           // [T][D] or null
  const _Float16 *s;         // [D] or null (backward)
  void *out;                 // [T][D]
  int T, D, k, E, slabs;
};

// Bound by HBM: 4096 tokens of 8 slots of 4096 in 95 us (6.3 TB/s), with plain loads of the rows,
// which nobody reads again, 126.
// out[t] = add[t] + s * sum of the token's rows, in the order of its slots (and for a slot of its
// slabs); four columns
// per thread.
template <bool BF>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs P) {
  const int quads = P.D / 4;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)P.T * quads) return;
  const int t = (int)(i / quads), d = (int)(i - (long long)t * quads) * 4;
  const int32_t *ids = P.ids + (size_t)t * P.k;
  const float *rows = P.part + (size_t)t * P.k * P.D + d;
  float4v y = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < P.k; j0 += 4) {
    float4v x[4];
    bool in[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = j0 + j < P.k ? ids[j0 + j] : -1;
      in[j] = e >= 0 && e < P.E;
      x[j] = float4v{0.f, 0.f, 0.f, 0.f};
      if (in[j]) x[j] = __builtin_nontemporal_load(reinterpret_cast<const float4v *>(rows + (size_t)(j0 + j) * P.D));
    }
    for (int i = 1; i < P.slabs; ++i) {
      const float *slab = rows + (size_t)i * P.T * P.k * P.D;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (in[j]) x[j] += __builtin_nontemporal_load(reinterpret_cast<const float4v *>(slab + (size_t)(j0 + j) * P.D));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) y += x[j];
  }
  if (P.s) {
#pragma unroll
    for (int v = 0; v < 4; ++v) y[v] *= (float)P.s[d + v];
  }
  const size_t at = (size_t)t * P.D + d;
  if (P.add) {
    const u16x4 a = *reinterpret_cast<const u16x4 *>(static_cast<const uint16_t *>(P.add) + at);
#pragma unroll
    for (int v = 0; v < 4; ++v) y[v] += act_to_f32<BF>(a[v]);
  }
  u16x4 out;
#pragma unroll
  for (int v = 0; v < 4; ++v) out[v] = f32_to_act<BF>(y[v]);
  *reinterpret_cast<u16x4 *>(static_cast<uint16_t *>(P.out) + at) = out;
}

// X * s, rounded once, eight columns per thread: an MFMA operand has 16 bits, and the product's other half
// would be a second MFMA for each.  The error of G and U goes from 2.1e-4 to 2.9e-4 (fp16) and from
// 1.66e-3 to 2.35e-3 (bf16), that of Y from 2.9e-4 to 4.2e-4 and from 2.35e-3 to 3.3e-3.
template <bool BF>
__global__ __launch_bounds__(256) void expert_prescale_kernel(const uint16_t *X, const _Float16 *s, uint16_t *out,
                                                              int K, long long octets) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= octets) return;
  const u32x4 x = *reinterpret_cast<const u32x4 *>(X + 8 * i);
  const half8 f = load_half8(s + (8 * i) % K);
  u32x4 y;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    y[q] = (uint32_t)f32_to_act<BF>(act_to_f32<BF>((uint16_t)x[q]) * (float)f[2 * q]) |
           (uint32_t)f32_to_act<BF>(act_to_f32<BF>((uint16_t)(x[q] >> 16)) * (float)f[2 * q + 1]) << 16;
  *reinterpret_cast<u32x4 *>(out + 8 * i) = y;
}

// ---- launches -----------------------------------------------------------------------------------

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// A call runs in rounds of at most this many slots, and of rows that 32-bit offsets reach,
// so that its workspace stays bounded.
constexpr long long kMaxSlots = 1 << 17;

// the most tiles that S slots can make
int max_tiles(int S, int E, int rows) { return std::min(S, S / rows + std::min(E, S)); }

int round_tokens(int T, int k, int D) {
  const long long by_slots = std::max<long long>(1, kMaxSlots / k);
  const long long by_bytes = std::max<long long>(1, ((1ll << 31) - 1) / (2ll * D));
  return (int)std::min<long long>(T, std::min(by_slots, by_bytes));
}

// Rows per tile, from the rows that an expert that is chosen at all gets on average.  Fewer
// rows than a tile has are loads and MFMAs of nothing; more are another reading of the
// weights, from the L2, and another decoding.  From 64 on a tile must also leave the
// first product (`columns` tiles wide) enough workgroups.  Times in us (bf16):
//   forward                          rows  8: 115 by 16, 109 by 32        rows 24: 152 by 32, 140 by 64
//   64 experts of 1024 x 4096        rows 48: 171 by 64, 202 by 128       rows 64: 229, 220; 512: 1222, 1061
//   8 of 14336 x 4096                rows  8: 209 by 16, 180 by 32        rows 24: 193 by 32, 245 by 64; 32: 252, 247
//                                    rows 48: 264 by 64, 332 by 128       rows 96: 429, 367; 512: 1698, 1494
//   16 of 1536 x 2048                rows 64: 59 by 32, 71 by 64          rows 192: 108 by 64, 117 by 128; 256: 141, 134
//   backward
//   64 experts of 1024 x 4096        rows  8: 131 by 16, 149 by 32        rows 12: 160, 156
//                                    rows 24: 190 by 32, 179 by 64        rows 48: 204 by 64, 229 by 128; 64: 260, 243
//   8 of 14336 x 4096                rows  8: 195 by 16, 217 by 32        rows 12: 248, 226
//                                    rows 24: 227 by 32, 265 by 64; 32: 348, 265
//                                    rows 48: 290 by 64, 343 by 128; 64: 426, 350
//   16 of 1536 x 2048                rows 64: 87 by 32, 90 by 64          rows 256: 156 by 64, 162 by 128; 512: 282, 259
// Slots that name no expert count in S, since the host cannot tell them: 512 slots of which 71 name one
// of 8 experts of 14336 x 4096 take 321 us, those 71 alone 168 (and a seventh of the workspace).
int tile_rows(int S, int E, int columns, int most16, int enough) {
  const long long chosen = std::min(E, S);
  if (S <= most16 * chosen) return 16;
  int rows = 32;
  if (S > 26 * chosen && (long long)max_tiles(S, E, 64) * columns >= enough) rows = 64;
  if (S > 56 * chosen && (long long)max_tiles(S, E, 128) * columns >= enough) rows = 128;
  return rows;
}
int forward_rows(int S, int E, int N) { return tile_rows(S, E, (N + 127) / 128, 6, 512); }
int backward_rows(int S, int E, int N) { return tile_rows(S, E, (N + 255) / 256, 10, 384); }

// Parts of the contraction of the product that makes the tokens' rows (D wide), each with its
// own workgroups and its own slab of sums, which combine_kernel adds.  The GPU holds 512
// workgroups at once.  Times of the whole call in us, with one, two and four parts:
//   forward, 8 experts of 14336 x 4096 (112 stages): 160 workgroups 237, 203, 180; 384: 583, 546, 533;
//   512: 758, 762, 777; 640: 1613, 1494, 1508
//   forward, 16 of 1536 x 2048 (12): 176: 43, 39, 41; 320: 55, 54, 61
//   backward, 8 of 14336 x 4096 (224): 160: 459, 286, 217; 384: 780, 701, 636; 512: 878, 880, 886;
//   640: 1835, 1600, 1577
//   backward, 16 of 1536 x 2048 (24): 224: 80, 72, 73; 384: 115, 111, 111; 640: 259, 261, 304
//   backward, 64 of 1024 x 4096 (16): 1152: 158, 165, 186
int row_slabs(int tiles, int D, int stages) {
  const long long units = (long long)tiles * ((D + 255) / 256);
  if (units < 512) return stages >= 64 ? 4 : stages >= 12 ? 2 : 1;
  return units > 512 && units <= 1280 && stages >= 64 ? 2 : 1;  // (a part's share of the last turn is smaller)
}

// Workgroups of the plan: one for each 2048 slots, at most 16.
unsigned plan_groups(int S) { return (unsigned)std::max(1, std::min(16, S / 2048)); }

// The workspace of one round.
struct Layout {
  int tokens, slots, rows, tiles, slabs;  // rows: per tile
  size_t order, list, count, xs, h, part, total;
};
Layout layout(const ExpertsDesc &d) {
  Layout l = {};
  l.tokens = round_tokens(d.T, d.k, d.D);
  l.slots = l.tokens * d.k;
  l.rows = forward_rows(l.slots, d.E, d.N);
  l.tiles = max_tiles(l.slots, d.E, l.rows);
  l.slabs = l.rows == 16 ? 1 : row_slabs(l.tiles, d.D, d.N / kGroup);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  l.order = take((size_t)l.slots * 4);
  l.list = take((size_t)l.tiles * sizeof(ExpertTile));
  l.count = take(4);
  l.xs = take(d.s ? (size_t)l.tokens * d.D * 2 : 0);
  l.h = take((size_t)l.slots * d.N * 2);
  l.part = take((size_t)l.slabs * l.slots * d.D * 4);
  l.total = at;
  return l;
}

// Streaming: 16-row blocks of the weights per workgroup, and waves that share a contraction.
// The more of both, the fewer times the activations are read and the fewer loads a
// wave waits for, but the fewer workgroups there are and the more the waves have to join.
// Times in us:
//   gate and up of 8 experts, 14336 x 4096, 2 slots: 46.7 by (4, 4), 52.0 by (4, 8), 44.8 by (4, 2);
//   of 64, 1024 x 4096, 8 slots 25.8, 25.3, 32.7; 128 slots 96, 110, 101
//   down of 8 experts, 4096 x 14336 (112 groups): 512 blocks over all tiles 46.5 by (2, 8), 63 by
//   (4, 4); 2048: 133 and 138; 2560: 181 and 172
//   down of 64, 4096 x 1024 (8 groups): 2048 blocks 24.6 by (4, 4), 25.7 by (4, 2), 25.8 by
//   (2, 8); 8192: 46, 44 and 64
struct StreamShape {
  int tn, ks;
};
StreamShape stream_shape(bool gated, int blocks, int groups, int tiles) {
  if (gated) return {4, 4};
  const bool many = (long long)tiles * blocks > 2048, deep = groups >= 32;
  if (many) return deep ? StreamShape{4, 4} : StreamShape{4, 2};
  return deep ? StreamShape{2, 8} : StreamShape{4, 4};
}

template <int EPI, bool GATHER, bool BF>
hipError_t launch_product(ExpertArgs a, int rows, int tiles, int slabs, hipStream_t stream) {
  const int blocks = (EPI == kGatedOut ? 2 : 1) * (a.N / kTileRows);
  if (rows == 16) {
    const StreamShape s = stream_shape(EPI == kGatedOut, blocks, a.K / kGroup, tiles);
    a.columns = (blocks + s.tn - 1) / s.tn;
    const dim3 grid((unsigned)((tiles * a.columns + 7) / 8 * 8)), threads(64 * s.ks);
#define W4_STREAM(TN, KS)                                                                        \
  if (s.tn == TN && s.ks == KS)                                                                  \
  hipLaunchKernelGGL((expert_stream_kernel<TN, KS, EPI, GATHER, BF>), grid, threads, 0, stream, a)
    W4_STREAM(4, 4);
    if constexpr (EPI == kRowsOut) {
      W4_STREAM(4, 2);
      W4_STREAM(2, 8);
    }
#undef W4_STREAM
  } else {
    a.columns = (blocks + 15) / 16;
    a.slabs = slabs;
    const dim3 grid((unsigned)((tiles * a.columns * slabs + 7) / 8 * 8));
    if (rows == 32)
      hipLaunchKernelGGL((expert_tile_kernel<2, EPI, GATHER, BF>), grid, dim3(256), 0, stream, a);
    else if (rows == 64)
      hipLaunchKernelGGL((expert_tile_kernel<4, EPI, GATHER, BF>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((expert_wide_kernel<EPI, GATHER, BF>), grid, dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

template <bool BF>
hipError_t launch_experts_typed(const ExpertsDesc &d, char *ws, hipStream_t stream) {
  const Layout l = layout(d);
  const size_t slot_n = (size_t)d.k * d.N * 2;
  for (int t0 = 0; t0 < d.T; t0 += l.tokens) {
    const int T = std::min(l.tokens, d.T - t0), S = T * d.k;
    const int32_t *ids = d.ids + (size_t)t0 * d.k;
    int32_t *order = reinterpret_cast<int32_t *>(ws + l.order), *count = reinterpret_cast<int32_t *>(ws + l.count);
    ExpertTile *list = reinterpret_cast<ExpertTile *>(ws + l.list);
    const bool small = S <= kSmallSlots && l.rows == 16;
    if (!small)
      hipLaunchKernelGGL(plan_kernel, dim3(plan_groups(S)), dim3(kPlanThreads), 0, stream, ids, S, d.E, l.rows, order, list, count);
    const char *X = static_cast<const char *>(d.X) + (size_t)t0 * d.D * 2;
    if (d.s) {
      const long long octets = (long long)T * d.D / 8;
      hipLaunchKernelGGL(expert_prescale_kernel<BF>, dim3((unsigned)((octets + 255) / 256)), dim3(256), 0, stream,
                         reinterpret_cast<const uint16_t *>(X), static_cast<const _Float16 *>(d.s),
                         reinterpret_cast<uint16_t *>(ws + l.xs), d.D, octets);
      X = ws + l.xs;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int tiles = max_tiles(S, d.E, l.rows);
    ExpertArgs a = {};
    a.plan = {small ? nullptr : order, list, count, ids, S, d.E};
    a.k = d.k;
    a.tokens = T;
    a.weights = d.weights + (size_t)t0 * d.k;
    a.act = d.act;
    auto weight = [&](int i, const ExpertWeight &w) {
      a.Wq[i] = static_cast<const uint8_t *>(w.Wq);
      a.scales[i] = static_cast<const _Float16 *>(w.scales);
      a.zeros[i] = static_cast<const _Float16 *>(w.zeros);
    };
    auto shape = [&](int N, int K) {
      a.N = N;
      a.K = K;
      a.code_bytes = (size_t)N * K / 2;
      a.meta_count = (size_t)N * meta_groups(K / kGroup);
    };
    weight(0, d.gate);
    weight(1, d.up);
    shape(d.N, d.D);
    a.A = X;
    a.s_down = static_cast<const _Float16 *>(d.s_down);
    a.G = d.G ? static_cast<char *>(d.G) + t0 * slot_n : nullptr;
    a.U = d.U ? static_cast<char *>(d.U) + t0 * slot_n : nullptr;
    a.H = ws + l.h;
    if ((e = launch_product<kGatedOut, true, BF>(a, l.rows, tiles, 1, stream)) != hipSuccess) return e;
    weight(0, d.down);
    shape(d.D, d.N);
    a.A = ws + l.h;
    a.part = reinterpret_cast<float *>(ws + l.part);
    if ((e = launch_product<kRowsOut, false, BF>(a, l.rows, tiles, l.slabs, stream)) != hipSuccess) return e;
    const size_t row = (size_t)t0 * d.D * 2;
    CombineArgs c = {};
    c.ids = ids;
    c.part = a.part;
    c.add = d.residual ? static_cast<const char *>(d.residual) + row : nullptr;
    c.out = static_cast<char *>(d.Y) + row;
    c.T = T;
    c.D = d.D;
    c.k = d.k;
    c.E = d.E;
    c.slabs = l.slabs;
    hipLaunchKernelGGL(combine_kernel<BF>, dim3((unsigned)(((long long)T * d.D / 4 + 255) / 256)), dim3(256), 0, stream, c);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---- backward launches

struct GradLayout {
  int tokens, slots, rows, tiles, columns, slabs;
  size_t order, list, count, dg, du, dw, part, total;
};
GradLayout grad_layout(const ExpertsGradDesc &d) {
  GradLayout l = {};
  l.tokens = round_tokens(d.T, d.k, d.D);
  l.slots = l.tokens * d.k;
  l.rows = backward_rows(l.slots, d.E, d.N);
  l.tiles = max_tiles(l.slots, d.E, l.rows);
  l.columns = (d.N + 255) / 256;
  l.slabs = row_slabs(l.tiles, d.D, 2 * (d.N / kGroup));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  l.order = take((size_t)l.slots * 4);
  l.list = take((size_t)l.tiles * sizeof(ExpertTile));
  l.count = take(4);
  l.dg = take((size_t)l.slots * d.N * 2);
  l.du = take((size_t)l.slots * d.N * 2);
  l.dw = take((size_t)l.slots * l.columns * 16);
  l.part = take((size_t)l.slabs * l.slots * d.D * 4);
  l.total = at;
  return l;
}

template <int EPI, bool GATHER, bool BF>
hipError_t launch_grad_product(ExpertGradArgs a, int rows, int tiles, int slabs, hipStream_t stream) {
  a.columns = (a.C + 255) / 256;
  a.slabs = slabs;
  const dim3 grid((unsigned)((tiles * a.columns * slabs + 7) / 8 * 8));
#define W4_GRAD(TM)                                                                              \
  if (rows == 16 * TM)                                                                           \
  hipLaunchKernelGGL((expert_grad_kernel<TM, EPI, GATHER, BF>), grid, dim3(256), 0, stream, a)
  W4_GRAD(1);
  W4_GRAD(2);
  W4_GRAD(4);
  W4_GRAD(8);
#undef W4_GRAD
  return hipGetLastError();
}

template <bool BF>
hipError_t launch_experts_grad_typed(const ExpertsGradDesc &d, char *ws, hipStream_t stream) {
  const GradLayout l = grad_layout(d);
  for (int t0 = 0; t0 < d.T; t0 += l.tokens) {
    const int T = std::min(l.tokens, d.T - t0), S = T * d.k;
    const int32_t *ids = d.ids + (size_t)t0 * d.k;
    int32_t *order = reinterpret_cast<int32_t *>(ws + l.order), *count = reinterpret_cast<int32_t *>(ws + l.count);
    ExpertTile *list = reinterpret_cast<ExpertTile *>(ws + l.list);
    hipLaunchKernelGGL(plan_kernel, dim3(plan_groups(S)), dim3(kPlanThreads), 0, stream, ids, S, d.E, l.rows, order, list, count);
    const int tiles = max_tiles(S, d.E, l.rows);
    const size_t row = (size_t)t0 * d.D * 2, slot_n = (size_t)t0 * d.k * d.N * 2;
    ExpertGradArgs a = {};
    a.plan = {order, list, count, ids, S, d.E};
    a.k = d.k;
    a.tokens = T;
    a.weights = d.weights + (size_t)t0 * d.k;
    a.act = d.act;
    a.code_bytes = (size_t)d.N * d.D / 2;
    a.meta_bytes = (size_t)(d.N / kGroup) * (d.D / kGroup) * kMetaBytes;
    a.A[0] = static_cast<const char *>(d.dY) + row;
    a.Wt[0] = static_cast<const uint8_t *>(d.down.Wt);
    a.meta[0] = static_cast<const uint8_t *>(d.down.meta);
    a.R = d.D;
    a.C = d.N;
    a.s_down = static_cast<const _Float16 *>(d.s_down);
    a.G = static_cast<const char *>(d.G) + slot_n;
    a.U = static_cast<const char *>(d.U) + slot_n;
    a.dG = ws + l.dg;
    a.dU = ws + l.du;
    a.dw_part = reinterpret_cast<float *>(ws + l.dw);
    hipError_t e = launch_grad_product<kActGradOut, true, BF>(a, l.rows, tiles, 1, stream);
    if (e != hipSuccess) return e;
    if (d.dweights)
      hipLaunchKernelGGL(weight_grad_kernel<BF>, dim3((unsigned)((S + 3) / 4)), dim3(256), 0, stream, ids, a.dw_part,
                         4 * l.columns, d.N / 64, S, d.E,
                         static_cast<char *>(d.dweights) + (size_t)t0 * d.k * (d.dweights_f32 ? 4 : 2), d.dweights_f32);
    if (d.dX) {
      a.A[0] = a.dG;
      a.A[1] = a.dU;
      a.Wt[0] = static_cast<const uint8_t *>(d.gate.Wt);
      a.Wt[1] = static_cast<const uint8_t *>(d.up.Wt);
      a.meta[0] = static_cast<const uint8_t *>(d.gate.meta);
      a.meta[1] = static_cast<const uint8_t *>(d.up.meta);
      a.R = d.N;
      a.C = d.D;
      a.part = reinterpret_cast<float *>(ws + l.part);
      if ((e = launch_grad_product<kGradRowsOut, false, BF>(a, l.rows, tiles, l.slabs, stream)) != hipSuccess) return e;
      CombineArgs c = {};
      c.ids = ids;
      c.part = a.part;
      c.add = d.add ? static_cast<const char *>(d.add) + row : nullptr;
      c.s = static_cast<const _Float16 *>(d.s);
      c.out = static_cast<char *>(d.dX) + row;
      c.T = T;
      c.D = d.D;
      c.k = d.k;
      c.E = d.E;
      c.slabs = l.slabs;
      hipLaunchKernelGGL(combine_kernel<BF>, dim3((unsigned)(((long long)T * d.D / 4 + 255) / 256)), dim3(256), 0, stream, c);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t experts_grad_workspace_bytes(const ExpertsGradDesc &d) { return d.T == 0 ? 0 : grad_layout(d).total; }

hipError_t launch_experts_grad(const ExpertsGradDesc &d, void *workspace, hipStream_t stream) {
  char *ws = static_cast<char *>(workspace);
  return d.bf16 ? launch_experts_grad_typed<true>(d, ws, stream) : launch_experts_grad_typed<false>(d, ws, stream);
}

size_t experts_workspace_bytes(const ExpertsDesc &d) { return d.T == 0 ? 0 : layout(d).total; }

hipError_t launch_experts(const ExpertsDesc &d, void *workspace, hipStream_t stream) {
  char *ws = static_cast<char *>(workspace);
  return d.bf16 ? launch_experts_typed<true>(d, ws, stream) : launch_experts_typed<false>(d, ws, stream);
}

}  // namespace w4a16
