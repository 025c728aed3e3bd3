// The norms before and after a block, with the block's gate and residual scale:
//   r = alpha * x + gate * post(y),   h = pre(r)
// y is the block's output, x the residual stream, post and pre one of
//   none   v
//   RMS    v * i * weight + bias,          i = 1 / sqrt(mean(v^2) + eps)
//   layer  (v - mean) * i * weight + bias, i = 1 / sqrt(mean((v - mean)^2) + eps)
// and its backward.  With n the normalised row, m(.) the mean over the row and
// d = weight * (gradient of the norm's output), the gradient of the norm's input is
//   RMS    i (d - n m(d n)),     layer  i (d - m(d) - n m(d n)).
//   R  = dr + pre'(dh; r),  dx = alpha R,  dgate = sum R post(y),  p = gate R,  dy = post'(p; y),
//   and the sums over rows of p n_y, p (post) and of dh n_r, dh (pre).
//
// Both are bound by HBM.  A row stays in registers from its one read to its one
// write: 8 or 16 columns per thread, 16-byte loads where rows are 16-byte aligned
// (D a multiple of 8), else one column at a time.  The mean is taken before the
// squared distances (two reductions, no bytes), so a large mean costs no precision.
// h is formed from the unrounded r; the backward normalises the r and y that it is
// given, and needs no saved statistics.
#include <algorithm>

#include "epilogue.h"
#include "w4a16_device.h"
#include "w4a16_internal.h"

namespace w4a16 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kNormNone = 0, kNormLayer = 2;

// v of the lane that the DPP control names, 0 where there is none
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}
// The wave's sum, in lane 63: prefix sums within rows of 16 lanes, then across the rows.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111, 0xf>(v);
  v += dpp<0x112, 0xf>(v);
  v += dpp<0x114, 0xf>(v);
  v += dpp<0x118, 0xf>(v);
  v += dpp<0x142, 0xa>(v);
  v += dpp<0x143, 0xc>(v);
  return v;
}

// The sums over the TPR threads of a row, in every one of them, in a fixed order.
// `red` holds one pair per wave and is not reused before two more barriers.
template <int TPR>
__device__ __forceinline__ void row_sum(float &a, float &b, float2 *red) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;
    const int wave = (threadIdx.x % TPR) >> 6;
    if ((threadIdx.x & 63) == 63) red[wave] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      a += red[w].x;
      b += red[w].y;
    }
  } else {
    a = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, a), 63));
    b = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, b), 63));
  }
}

// CPT columns of one row per thread, as raw 16-bit values: 8 consecutive ones at
// 8 (t + TPR i), or single ones at t + TPR i.  Columns from D on read as 0.
template <int TPR, int CPT, bool VEC>
struct Row {
  uint32_t w[CPT / 2];

  static __device__ __forceinline__ int column(int t, int i) {
    return VEC ? 8 * (t + TPR * (i / 8)) + i % 8 : t + TPR * i;
  }
  __device__ __forceinline__ void load(const uint16_t *row, int t, int D) {
    if constexpr (VEC) {
#pragma unroll
      for (int g = 0; g < CPT / 8; ++g) {
        const int c = 8 * (t + TPR * g);
        u32x4 v = {0, 0, 0, 0};
        if (c < D) v = *reinterpret_cast<const u32x4 *>(row + c);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[4 * g + q] = v[q];
      }
    } else {
#pragma unroll
      for (int i = 0; i < CPT; i += 2) {
        const int c0 = t + TPR * i, c1 = c0 + TPR;
        w[i / 2] = (c0 < D ? row[c0] : 0u) | (c1 < D ? (uint32_t)row[c1] << 16 : 0u);
      }
    }
  }
  __device__ __forceinline__ void store(uint16_t *row, int t, int D) const {
    if constexpr (VEC) {
#pragma unroll
      for (int g = 0; g < CPT / 8; ++g) {
        const int c = 8 * (t + TPR * g);
        const u32x4 v = {w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]};
        if (c < D) *reinterpret_cast<u32x4 *>(row + c) = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int c = t + TPR * i;
        if (c < D) row[c] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
      }
    }
  }
  template <bool BF>
  __device__ __forceinline__ float get(int i) const {
    return act_to_f32<BF>((uint16_t)(w[i / 2] >> (16 * (i & 1))));
  }
  template <bool BF>
  __device__ __forceinline__ void set(int i, float v) {  // i even first, then i + 1
    const uint32_t h = f32_to_act<BF>(v);
    w[i / 2] = i & 1 ? w[i / 2] | h << 16 : h;
  }
};

// Which of them there are; FULL: all (D = TPR * CPT), known when compiling.
template <int TPR, int CPT, bool VEC, bool FULL = false>
struct Columns {
  bool in[VEC ? CPT / 8 : CPT];
  __device__ __forceinline__ Columns(int t, int D) {
#pragma unroll
    for (int i = 0; i < (VEC ? CPT / 8 : CPT); ++i)
      in[i] = FULL || Row<TPR, CPT, VEC>::column(t, VEC ? 8 * i : i) < D;
  }
  __device__ __forceinline__ bool operator[](int i) const { return FULL || in[VEC ? i / 8 : i]; }
};

// v becomes its normalised row
template <int TPR, int CPT, bool VEC>
__device__ __forceinline__ void normalize(float (&v)[CPT], const Columns<TPR, CPT, VEC> &in, int D,
                                          bool layer, float eps, float2 *red) {
  float a = 0.f, b = 0.f;
  if (layer) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) a += v[i];
    row_sum<TPR>(a, b, red);
    const float mean = a / D;
#pragma unroll
    for (int i = 0; i < CPT; ++i) v[i] = in[i] ? v[i] - mean : 0.f;
    a = b = 0.f;
  }
#pragma unroll
  for (int i = 0; i < CPT; ++i) a = __builtin_fmaf(v[i], v[i], a);
  row_sum<TPR>(a, b, red + TPR / 64);
  const float inv = rsqrtf(a / D + eps);
#pragma unroll
  for (int i = 0; i < CPT; ++i) v[i] *= inv;
}

template <int TPR, int CPT, bool BF, bool VEC>
__device__ __forceinline__ void affine(float (&v)[CPT], const void *weight, const void *bias, int t,
                                       int D) {
  Row<TPR, CPT, VEC> p;
  if (weight) {
    p.load(static_cast<const uint16_t *>(weight), t, D);
#pragma unroll
    for (int i = 0; i < CPT; ++i) v[i] *= p.template get<BF>(i);
  }
  if (bias) {
    p.load(static_cast<const uint16_t *>(bias), t, D);
#pragma unroll
    for (int i = 0; i < CPT; ++i) v[i] += p.template get<BF>(i);
  }
}

// One row per TPR threads.  One row of 4096: 2.9 us, which is a launch and two
// reductions; 4096 x 8192 with both norms (bf16): 41.3-41.7 us, 6.4 TB/s of what it reads and writes.
template <int TPR, int CPT, bool BF, bool VEC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormDesc P) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  __shared__ float2 red[4 * TPR / 64];
  const int t = threadIdx.x % TPR, D = P.D;
  const long long m = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
  if (kRows > 1 && m >= P.T) return;  // (whole waves: rows of more than one are a workgroup each)
  const Columns<TPR, CPT, VEC> in(t, D);
  const size_t at = (size_t)m * D;
  Row<TPR, CPT, VEC> io, iy, ig;
  io.load(static_cast<const uint16_t *>(P.x) + at, t, D);
  if (P.y) iy.load(static_cast<const uint16_t *>(P.y) + at, t, D);
  float r[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) r[i] = P.alpha * io.template get<BF>(i);
  if (P.y) {
    if (P.gate) ig.load(static_cast<const uint16_t *>(P.gate) + (size_t)(m / P.gate_rows) * D, t, D);
    float y[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) y[i] = iy.template get<BF>(i);
    if (P.post.kind != kNormNone) {
      normalize<TPR, CPT, VEC>(y, in, D, P.post.kind == kNormLayer, P.post.eps, red);
      affine<TPR, CPT, BF, VEC>(y, P.post.weight, P.post.bias, t, D);
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i)
      r[i] = P.gate ? __builtin_fmaf(ig.template get<BF>(i), y[i], r[i]) : r[i] + y[i];
  }
  if (P.r) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) io.template set<BF>(i, r[i]);
    io.store(static_cast<uint16_t *>(P.r) + at, t, D);
  }
  if (P.h) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) r[i] = in[i] ? r[i] : 0.f;
    normalize<TPR, CPT, VEC>(r, in, D, P.pre.kind == kNormLayer, P.pre.eps, red + 2 * TPR / 64);
    affine<TPR, CPT, BF, VEC>(r, P.pre.weight, P.pre.bias, t, D);
#pragma unroll
    for (int i = 0; i < CPT; ++i) io.template set<BF>(i, r[i]);
    io.store(static_cast<uint16_t *>(P.h) + at, t, D);
  }
}

// ---- backward -----------------------------------------------------------------------

// The sums over rows that a call may want.
enum { kSumGate = 0, kSumPostW, kSumPostB, kSumPreW, kSumPreB };

// What the sums' kernel needs of a row whose activations' gradients are done:
// R = dr + inv_r (w dh - a - n b), n = (r - mean_r) inv_r.
struct RowStats {
  float mean_r, inv_r, a, b, mean_y, inv_y;
};

struct NormGradArgs {
  NormGradDesc d;
  float *part[kNormSums];  // the strips' sums [strips][D], or null
  RowStats *stats;         // null: the sums are taken in norm_grad_kernel
  int rows;                // rows per strip
  int per_segment;         // strips per gate vector (0: a strip is whole segments)
};

// The rows of strip `block`.
__device__ __forceinline__ void strip_rows(const NormGradArgs &A, int block, int &m0, int &m1) {
  const NormGradDesc &P = A.d;
  if (A.per_segment) {
    const int seg = block / A.per_segment;
    const long long first = (long long)seg * P.gate_rows;
    const long long at = first + (long long)(block - seg * A.per_segment) * A.rows;
    m0 = (int)std::min(at, (long long)P.T);
    m1 = (int)std::min(std::min(at + A.rows, first + P.gate_rows), (long long)P.T);
  } else {
    m0 = (int)std::min((long long)block * A.rows, (long long)P.T);
    m1 = (int)std::min((long long)m0 + A.rows, (long long)P.T);
  }
}

// The call's arguments, read again where they are used: kept in registers through
// the row loop, its pointers alone would take most of the scalar ones.
__device__ __forceinline__ const NormGradArgs &args_again() {
  typedef const __attribute__((address_space(4))) NormGradArgs *Arg;
  uint64_t p = reinterpret_cast<uint64_t>((Arg)__builtin_amdgcn_kernarg_segment_ptr());
  asm volatile("" : "+s"(p));
  return *(const NormGradArgs *)reinterpret_cast<Arg>(p);
}

// Bound by HBM, and at this occupancy (four waves per SIMD, of 128 registers) by a row's four
// reductions in turn: 4092 x 4096 with layer norms and gates (bf16), 201 MB and 42 of the
// strips' sums, takes 58-63 us (3.9-4.2 TB/s).
// SUMS: a strip of rows per workgroup, one row at a time with the next one's loads in
// flight.  A thread keeps its columns' sums over the strip, so the sums cost one
// fp32 row per strip; norm_sum_kernel adds the strips in order.
// Without: one row per workgroup (strips of one row), which leaves its statistics.
template <int TPR, int CPT, bool BF, bool VEC, bool SUMS, bool FULL = false>
__global__ __launch_bounds__(TPR) void norm_grad_kernel(NormGradArgs A0) {
  typedef Row<TPR, CPT, VEC> R16;
  constexpr int kW = TPR / 64;
  __shared__ float2 red[4 * kW];
  const int t = threadIdx.x, D = FULL ? TPR * CPT : A0.d.D;
  const float rD = 1.0f / D;
  const Columns<TPR, CPT, VEC, FULL> in(t, D);
  const bool pre = A0.d.pre.kind != kNormNone, post = A0.d.post.kind != kNormNone;
  const bool pre_layer = A0.d.pre.kind == kNormLayer, post_layer = A0.d.post.kind == kNormLayer;
  int m0 = blockIdx.x, m1 = blockIdx.x + 1;
  if (SUMS) strip_rows(A0, blockIdx.x, m0, m1);
  float s_gate[CPT], s_pw[CPT], s_pb[CPT], s_rw[CPT], s_rb[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) s_gate[i] = s_pw[i] = s_pb[i] = s_rw[i] = s_rb[i] = 0.f;

  struct In {
    R16 dr, dh, y, r;
  };
  auto load = [&](int m, In &v) {
    const NormGradDesc &P = args_again().d;
    const size_t at = (size_t)m * D;
    if (P.dr) v.dr.load(static_cast<const uint16_t *>(P.dr) + at, t, D);
    if (P.y) v.y.load(static_cast<const uint16_t *>(P.y) + at, t, D);
    if (pre) {
      v.dh.load(static_cast<const uint16_t *>(P.dh) + at, t, D);
      v.r.load(static_cast<const uint16_t *>(P.r) + at, t, D);
    }
  };
  constexpr bool kAhead = SUMS && CPT == 8;  // (16 columns leave no registers for the next row)
  In cur, nxt;
  if (kAhead && m0 < m1) load(m0, cur);
  for (int m = m0; m < m1; ++m) {
    if (!kAhead)
      load(m, cur);
    else if (m + 1 < m1)
      load(m + 1, nxt);
    const NormGradArgs &A = args_again();
    const NormGradDesc &P = A.d;
    const size_t at = (size_t)m * D;
    float mean_r = 0.f, mean_y = 0.f;
    if (pre_layer || post_layer) {
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        if (pre_layer) a += cur.r.template get<BF>(i);
        if (post_layer) b += cur.y.template get<BF>(i);
      }
      row_sum<TPR>(a, b, red);
      mean_r = a * rD;
      mean_y = b * rD;
    }
    auto r_at = [&](int i) { return in[i] ? cur.r.template get<BF>(i) - mean_r : 0.f; };
    auto y_at = [&](int i) { return in[i] ? cur.y.template get<BF>(i) - mean_y : 0.f; };
    float inv_r = 0.f, inv_y = 1.f;
    if (pre || post) {
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        if (pre) {
          const float v = r_at(i);
          a = __builtin_fmaf(v, v, a);
        }
        if (post) {
          const float v = y_at(i);
          b = __builtin_fmaf(v, v, b);
        }
      }
      row_sum<TPR>(a, b, red + kW);
      if (pre) inv_r = rsqrtf(a * rD + P.pre.eps);
      if (post) inv_y = rsqrtf(b * rD + P.post.eps);
    }
    float g[CPT];  // R
    float pa = 0.f, pb = 0.f;
    if (pre) {
      R16 w;
      if (P.pre.weight) w.load(static_cast<const uint16_t *>(P.pre.weight), t, D);
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const float dh = cur.dh.template get<BF>(i), n = r_at(i) * inv_r;
        if (SUMS) {
          s_rw[i] = __builtin_fmaf(dh, n, s_rw[i]);
          s_rb[i] += dh;
        }
        g[i] = P.pre.weight ? dh * w.template get<BF>(i) : dh;
        pa += g[i];
        pb = __builtin_fmaf(g[i], n, pb);
      }
      row_sum<TPR>(pa, pb, red + 2 * kW);
      pa = pre_layer ? pa * rD : 0.f;
      pb *= rD;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        g[i] = inv_r * (g[i] - pa - r_at(i) * inv_r * pb);
        if (P.dr) g[i] += cur.dr.template get<BF>(i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < CPT; ++i) g[i] = cur.dr.template get<BF>(i);
    }
    R16 out;
    if (P.dx) {
      const float alpha = P.alpha;
#pragma unroll
      for (int i = 0; i < CPT; ++i) out.template set<BF>(i, alpha * g[i]);
      out.store(static_cast<uint16_t *>(P.dx) + at, t, D);
    }
    if (P.y) {
      R16 w;
      if (post && P.post.weight) w.load(static_cast<const uint16_t *>(P.post.weight), t, D);
      if (P.gate) {
        R16 v16;
        if (SUMS && A.part[kSumGate]) {
          if (post && P.post.bias) v16.load(static_cast<const uint16_t *>(P.post.bias), t, D);
#pragma unroll
          for (int i = 0; i < CPT; ++i) {
            float v = y_at(i) * inv_y;
            if (post && P.post.weight) v *= w.template get<BF>(i);
            if (post && P.post.bias) v += v16.template get<BF>(i);
            s_gate[i] = __builtin_fmaf(g[i], v, s_gate[i]);
          }
        }
        v16.load(static_cast<const uint16_t *>(P.gate) + (size_t)(m / P.gate_rows) * D, t, D);
#pragma unroll
        for (int i = 0; i < CPT; ++i) g[i] *= v16.template get<BF>(i);
      }
      if (post) {
        float a = 0.f, c = 0.f;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          const float n = y_at(i) * inv_y;
          if (SUMS) {
            s_pw[i] = __builtin_fmaf(g[i], n, s_pw[i]);
            s_pb[i] += g[i];
          }
          if (P.post.weight) g[i] *= w.template get<BF>(i);
          if (!in[i]) g[i] = 0.f;
          a += g[i];
          c = __builtin_fmaf(g[i], n, c);
        }
        row_sum<TPR>(a, c, red + 3 * kW);
        a = post_layer ? a * rD : 0.f;
        c *= rD;
#pragma unroll
        for (int i = 0; i < CPT; ++i) g[i] = inv_y * (g[i] - a - y_at(i) * inv_y * c);
      }
      if (P.dy) {
#pragma unroll
        for (int i = 0; i < CPT; ++i) out.template set<BF>(i, g[i]);
        out.store(static_cast<uint16_t *>(P.dy) + at, t, D);
      }
      // a strip of whole segments: the segment's gradient is complete with its last row
      if (SUMS && P.gate && A.part[kSumGate] && !A.per_segment &&
          (m + 1 == m1 || (m + 1) % P.gate_rows == 0)) {
        float *dst = A.part[kSumGate] + (size_t)(m / P.gate_rows) * D;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          if (in[i]) dst[R16::column(t, i)] = s_gate[i];
          s_gate[i] = 0.f;
        }
      }
    }
    if (!SUMS && A.stats && t == 0) A.stats[m] = {mean_r, inv_r, pa, pb, mean_y, inv_y};
    if constexpr (kAhead) cur = nxt;
  }
  if constexpr (SUMS) {
    auto put = [&](int which, const float (&s)[CPT]) {
      float *dst = args_again().part[which];
      if (!dst) return;
      dst += (size_t)blockIdx.x * D;
#pragma unroll
      for (int i = 0; i < CPT; ++i)
        if (in[i]) dst[R16::column(t, i)] = s[i];
    };
    if (A0.per_segment) put(kSumGate, s_gate);
    put(kSumPostW, s_pw);
    put(kSumPostB, s_pb);
    put(kSumPreW, s_rw);
    put(kSumPreB, s_rb);
  }
}

// The sums of a strip of rows, COLS columns per thread, from the rows' statistics: rows
// of more than 8192 columns, whose sums do not fit in registers beside the row, and
// rows that are not read in 16-byte pieces (one column per thread, else four).  It reads once
// more what the rows' kernel read: the backward of 2048 x 12288 (RMS norms, bf16) takes 124 us,
// 80 of them without the sums; with one column per thread there too 169.
template <bool BF, int COLS>
__global__ __launch_bounds__(256) void norm_strip_kernel(NormGradArgs A) {
  typedef uint16_t Piece __attribute__((ext_vector_type(COLS)));
  const NormGradDesc &P = A.d;
  const int D = P.D, blocks = (D + 256 * COLS - 1) / (256 * COLS);
  const int strip = (int)blockIdx.x / blocks, n = (((int)blockIdx.x - strip * blocks) * 256 + threadIdx.x) * COLS;
  if (n >= D) return;
  int m0, m1;
  strip_rows(A, strip, m0, m1);
  struct Values {
    float v[COLS];
  };
  auto load = [&](const void *p, size_t at) {
    const Piece x = *reinterpret_cast<const Piece *>(static_cast<const uint16_t *>(p) + at);
    Values o;
#pragma unroll
    for (int i = 0; i < COLS; ++i) o.v[i] = act_to_f32<BF>(x[i]);
    return o;
  };
  auto or_else = [&](bool there, const void *p, float other) {
    if (there && p) return load(p, n);
    Values o;
#pragma unroll
    for (int i = 0; i < COLS; ++i) o.v[i] = other;
    return o;
  };
  const bool pre = P.pre.kind != kNormNone, post = P.post.kind != kNormNone;
  const Values wr = or_else(pre, P.pre.weight, 1.f), wy = or_else(post, P.post.weight, 1.f), by = or_else(post, P.post.bias, 0.f);
  float s_gate[COLS], s_pw[COLS], s_pb[COLS], s_rw[COLS], s_rb[COLS];
#pragma unroll
  for (int i = 0; i < COLS; ++i) s_gate[i] = s_pw[i] = s_pb[i] = s_rw[i] = s_rb[i] = 0.f;
  auto put = [&](float *dst, const float (&v)[COLS]) {
#pragma unroll
    for (int i = 0; i < COLS; ++i) dst[i] = v[i];
  };
#pragma unroll 4
  for (int m = m0; m < m1; ++m) {
    const size_t at = (size_t)m * D + n;
    const RowStats q = A.stats[m];
    Values R = {};
    if (P.dr) R = load(P.dr, at);
    if (pre) {
      const Values dh = load(P.dh, at), r = load(P.r, at);
#pragma unroll
      for (int i = 0; i < COLS; ++i) {
        const float x = (r.v[i] - q.mean_r) * q.inv_r;
        s_rw[i] = __builtin_fmaf(dh.v[i], x, s_rw[i]);
        s_rb[i] += dh.v[i];
        R.v[i] += q.inv_r * (dh.v[i] * wr.v[i] - q.a - x * q.b);
      }
    }
    if (P.y) {
      const Values y = load(P.y, at);
      Values gate;
      if (P.gate) gate = load(P.gate, (size_t)(m / P.gate_rows) * D + n);
#pragma unroll
      for (int i = 0; i < COLS; ++i) {
        const float x = (y.v[i] - q.mean_y) * q.inv_y;
        if (P.gate) {
          s_gate[i] = __builtin_fmaf(R.v[i], __builtin_fmaf(x, wy.v[i], by.v[i]), s_gate[i]);
          R.v[i] *= gate.v[i];
        }
        s_pw[i] = __builtin_fmaf(R.v[i], x, s_pw[i]);
        s_pb[i] += R.v[i];
      }
      if (P.gate && A.part[kSumGate] && !A.per_segment && (m + 1 == m1 || (m + 1) % P.gate_rows == 0)) {
        put(A.part[kSumGate] + (size_t)(m / P.gate_rows) * D + n, s_gate);
#pragma unroll
        for (int i = 0; i < COLS; ++i) s_gate[i] = 0.f;
      }
    }
  }
  const size_t to = (size_t)strip * D + n;
  if (A.per_segment && A.part[kSumGate]) put(A.part[kSumGate] + to, s_gate);
  if (A.part[kSumPostW]) put(A.part[kSumPostW] + to, s_pw);
  if (A.part[kSumPostB]) put(A.part[kSumPostB] + to, s_pb);
  if (A.part[kSumPreW]) put(A.part[kSumPreW] + to, s_rw);
  if (A.part[kSumPreB]) put(A.part[kSumPreB] + to, s_rb);
}

// out[i][n] = the sum over its strips of part[(i * strips + k)][n], for the sums of a
// backward call: 8 lanes per column, each over every 8th strip, then the lanes in order.
struct NormSumItem {
  const float *part;
  float *out;
  int strips, segments, block0;
};
struct NormSumArgs {
  NormSumItem s[kNormSums];
  int count, D;
};
__global__ __launch_bounds__(256) void norm_sum_kernel(NormSumArgs A) {
  int si = 0;
#pragma unroll
  for (int i = 1; i < kNormSums; ++i)
    if (i < A.count && (int)blockIdx.x >= A.s[i].block0) si = i;
  const NormSumItem &S = A.s[si];
  const int blocks = (A.D + 31) / 32, local = (int)blockIdx.x - S.block0;
  const int seg = local / blocks, x = threadIdx.x & 31, lane = threadIdx.x >> 5;
  const int n = (local - seg * blocks) * 32 + x;
  float s = 0.f;
  if (n < A.D) {
    const float *src = S.part + (size_t)seg * S.strips * A.D + n;
#pragma unroll 4
    for (int k = lane; k < S.strips; k += 8) s += src[(size_t)k * A.D];
  }
  __shared__ float red[8][32];
  red[lane][x] = s;
  __syncthreads();
  if (lane == 0 && n < A.D) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][x];
    S.out[(size_t)seg * A.D + n] = s;
  }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Strips of a backward call: about 2^18 threads of them (four waves per SIMD), of at
// least 8 rows; within one gate vector's rows each, or of whole ones.  The backward of
// 4092 x 4096 (layer norms and four gates, bf16) takes 58 to 63 + 8 us so, and with half as
// many strips 75 + 5 (two rows at a time there, for 176 registers: 73 + 5).
struct NormPlan {
  bool fused;  // the sums are taken where the rows are
  int tpr, cpt;
  int rows, per_segment, strips, segments;
};
NormPlan plan_norm_grad(const NormGradDesc &d) {
  NormPlan p = {};
  p.fused = d.D % 8 == 0 && d.D <= 8192;
  p.tpr = 64;
  while (p.tpr * 8 < d.D && p.tpr < 512) p.tpr *= 2;
  p.cpt = d.D <= 4096 ? 8 : 16;
  const long long T = d.T, gr = d.gate ? d.gate_rows : T;
  const long long want = std::max(1, (1 << 18) / p.tpr);
  const long long rows = std::max<long long>(8, (T + want - 1) / want);
  p.segments = (int)((T + gr - 1) / gr);
  if (gr > rows) {
    const long long per = (gr + rows - 1) / rows;
    p.per_segment = (int)per;
    p.rows = (int)((gr + per - 1) / per);
    p.strips = (int)(per * p.segments);
  } else {
    p.rows = (int)(rows / gr * gr);
    p.strips = (int)((T + p.rows - 1) / p.rows);
  }
  return p;
}

bool any_sum(const NormGradDesc &d) {
  return std::any_of(d.sums, d.sums + kNormSums, [](const void *s) { return s != nullptr; });
}

template <bool BF, bool VEC>
void launch_norm_typed(const NormDesc &d, hipStream_t stream) {
#define W4_NORM(TPR, CPT)                                                                        \
  hipLaunchKernelGGL((norm_kernel<TPR, CPT, BF, VEC>),                                           \
                     dim3((unsigned)((d.T + (TPR < 256 ? 256 / TPR : 1) - 1) / (TPR < 256 ? 256 / TPR : 1))), \
                     dim3(TPR < 256 ? 256 : TPR), 0, stream, d)
  if (d.D <= 64 * 8)
    W4_NORM(64, 8);
  else if (d.D <= 256 * 8)
    W4_NORM(256, 8);
  else if (d.D <= 256 * 16)
    W4_NORM(256, 16);
  else if (d.D <= 512 * 16)
    W4_NORM(512, 16);
  else
    W4_NORM(1024, 16);
#undef W4_NORM
}

template <bool BF>
void launch_norm_grad_fused(const NormPlan &p, const NormGradArgs &a, hipStream_t stream) {
#define W4_NORM(TPR, CPT)                                                                        \
  if (p.tpr == TPR && p.cpt == CPT) {                                                            \
    if (a.d.D == TPR * CPT)                                                                      \
      hipLaunchKernelGGL((norm_grad_kernel<TPR, CPT, BF, true, true, true>),                     \
                         dim3((unsigned)p.strips), dim3(TPR), 0, stream, a);                     \
    else                                                                                         \
      hipLaunchKernelGGL((norm_grad_kernel<TPR, CPT, BF, true, true>), dim3((unsigned)p.strips), \
                         dim3(TPR), 0, stream, a);                                               \
  }
  W4_NORM(64, 8)
  W4_NORM(128, 8)
  W4_NORM(256, 8)
  W4_NORM(512, 8)
  W4_NORM(512, 16)
#undef W4_NORM
}

template <bool BF, bool VEC>
void launch_norm_grad_rows(const NormGradArgs &a, hipStream_t stream) {
  const int D = a.d.D;
#define W4_NORM(TPR, CPT)                                                                        \
  hipLaunchKernelGGL((norm_grad_kernel<TPR, CPT, BF, VEC, false>), dim3((unsigned)a.d.T),        \
                     dim3(TPR), 0, stream, a)
  if constexpr (!VEC) {  // (shorter rows of 16-byte pieces take the sums along)
    if (D <= 64 * 8) {
      W4_NORM(64, 8);
      return;
    }
    if (D <= 512 * 8) {
      W4_NORM(512, 8);
      return;
    }
  }
  W4_NORM(1024, 16);
#undef W4_NORM
}

}  // namespace

hipError_t launch_norm(const NormDesc &d, hipStream_t stream) {
  if (d.T == 0) return hipSuccess;
  if (d.bf16) {
    d.D % 8 == 0 ? launch_norm_typed<true, true>(d, stream) : launch_norm_typed<true, false>(d, stream);
  } else {
    d.D % 8 == 0 ? launch_norm_typed<false, true>(d, stream) : launch_norm_typed<false, false>(d, stream);
  }
  return hipGetLastError();
}

size_t norm_grad_workspace_bytes(const NormGradDesc &d) {
  if (d.T == 0 || !any_sum(d)) return 0;
  const NormPlan p = plan_norm_grad(d);
  size_t n = p.fused ? 0 : align256((size_t)d.T * sizeof(RowStats));
  for (int i = 0; i < kNormSums; ++i)
    if (d.sums[i] && !(i == kSumGate && !p.per_segment))
      n += align256((size_t)p.strips * d.D * sizeof(float));
  return n;
}

// (T = 0: the sums are over no rows, zeros)
hipError_t launch_norm_grad(const NormGradDesc &d, void *workspace, hipStream_t stream) {
  NormPlan p = {};
  if (d.T > 0) p = plan_norm_grad(d);
  NormGradArgs a = {};
  a.d = d;
  a.rows = p.rows;
  a.per_segment = p.per_segment;
  char *ws = static_cast<char *>(workspace);
  if (d.T > 0 && !p.fused && any_sum(d)) {
    a.stats = reinterpret_cast<RowStats *>(ws);
    ws += align256((size_t)d.T * sizeof(RowStats));
  }
  NormSumArgs sums = {};
  sums.D = d.D;
  int block = 0;
  for (int i = 0; i < kNormSums; ++i) {
    if (!d.sums[i]) continue;
    if (i == kSumGate && !p.per_segment) {  // whole segments: written where they end
      a.part[i] = static_cast<float *>(d.sums[i]);
      continue;
    }
    if (d.T > 0) {
      a.part[i] = reinterpret_cast<float *>(ws);
      ws += align256((size_t)p.strips * d.D * sizeof(float));
    }
    const int segments = i == kSumGate ? p.segments : 1;
    sums.s[sums.count++] = {a.part[i], static_cast<float *>(d.sums[i]),
                            i == kSumGate ? p.per_segment : p.strips, segments, block};
    block += segments * ((d.D + 31) / 32);
  }
  if (d.T > 0) {
    if (p.fused) {
      d.bf16 ? launch_norm_grad_fused<true>(p, a, stream) : launch_norm_grad_fused<false>(p, a, stream);
    } else if (d.D % 8 == 0) {
      d.bf16 ? launch_norm_grad_rows<true, true>(a, stream) : launch_norm_grad_rows<false, true>(a, stream);
    } else {
      d.bf16 ? launch_norm_grad_rows<true, false>(a, stream) : launch_norm_grad_rows<false, false>(a, stream);
    }
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.stats) {
#define W4_STRIP(BF, COLS)                                                                        \
  hipLaunchKernelGGL((norm_strip_kernel<BF, COLS>),                                               \
                     dim3((unsigned)(p.strips * ((d.D + 256 * COLS - 1) / (256 * COLS)))), dim3(256), 0, stream, a)
      if (d.D % 8 == 0) {
        if (d.bf16)
          W4_STRIP(true, 4);
        else
          W4_STRIP(false, 4);
      } else if (d.bf16) {
        W4_STRIP(true, 1);
      } else {
        W4_STRIP(false, 1);
      }
#undef W4_STRIP
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
  }
  if (sums.count)
    hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)block), dim3(256), 0, stream, sums);
  return hipGetLastError();
}

}  // namespace w4a16
