// norm.hip — RMS norm with the residual's addition and a block-scaled output, and its backward
// pass, for gfx950.
//
// Forward, per row:  s = x + r (fp32, rounded to the tensors' type: the residual stream that is
// stored is the value that is normalised, so the backward pass and a recomputation from the
// stored sum see the same numbers),  rho = 1 / sqrt(mean(s^2) + eps),  y = s rho g.
// The sum of squares and rho are formed in 64 bits and y as an unevaluated sum of two fp32 values
// (2^-45 of it), and every output is rounded from that once (round_odd). So the outputs do not
// depend on the order of the sum, that is on the launch shape or on how many rows share the call,
// and the codes are those of the definition in 64 bits.
// Backward:  u = dy g, z = s rho, c = mean(u z):  dx = rho (u - z c) (+ dsum),  dg = sum_rows dy z.
#include "mx_device.h"
#include "mx_launch.h"

#include <type_traits>

using namespace mxd;

namespace {

// threads of a grid: 12 waves a SIMD of 256 compute units, two to three times what they hold, which
// evens out the workgroups' ends (262144 rows of 128: 25.4 us, 27.9 with 6 waves, 31.0 with 4;
// 8192 x 4096: 58.0, 60.4 and 58.5)
constexpr int64_t kNormThreads = 256 * 12 * 4 * 64;

// 8 values of a row chunk
template <bool BF16>
__device__ __forceinline__ void load_chunk(const void* p, int64_t off, float (&v)[8]) {
  if constexpr (BF16) {
    widen_bf16x8(*reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(p) + off), v);
  } else {
    const f32x4* q = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + off);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = a[k];
      v[4 + k] = b[k];
    }
  }
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ u32x4 pack_bf16x8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x2_t p = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};  // nearest even
    w[i] = __builtin_bit_cast(uint32_t, p);
  }
  return u32x4{w[0], w[1], w[2], w[3]};
}

__device__ __forceinline__ void load_gamma(const void* g, bool bf16, int64_t off, float (&v)[8]) {
  if (bf16) load_chunk<true>(g, off, v);
  else load_chunk<false>(g, off, v);
}

// s rho g as hi + lo: products with their rounding errors, which the fused multiply-add gives
// exactly. |lo| is at most a few half steps of hi; what is dropped is 2^-47 of the product (more
// where errors fall below fp32's range: |y| under 2^-100; rho is kept within 2^-90 .. 2^90).
__device__ __forceinline__ void product(float s, float rho, float rho_lo, float g, float& hi,
                                        float& lo) {
  const float p = s * rho;
  const float pe = fmaf(s, rho_lo, fmaf(s, rho, -p));
  hi = p * g;
  lo = fmaf(pe, g, fmaf(p, g, -hi));
}

// hi + lo to nearest; a zero keeps the sign of hi (codes carry it), where -0 + 0 would be +0. Where
// hi is infinite, lo is the opposite infinity and the sum a NaN: see nearest.
__device__ __forceinline__ float sum_of(float hi, float lo) {
  return __builtin_copysignf(hi + lo, hi);
}
__device__ __forceinline__ float nearest(float hi, float lo) {
  return fabsf(hi) < __builtin_inff() ? sum_of(hi, lo) : hi;
}

// hi + lo in fp32 by rounding to odd: of the two fp32 values around an inexact sum the one whose
// last bit is set. A rounding of the result to at most 22 significant bits (bf16, E4M3, E5M2,
// E2M1, the thresholds of the stochastic rounding, the block maximum's exponent) is then the
// rounding of hi + lo itself: no tie is made or lost on the way. Infinities and NaNs stay such.
__device__ __forceinline__ float round_odd(float hi, float lo) {
  const float h = nearest(hi, lo);
  const float l = lo - (h - hi);  // exact: |lo| <= |hi|
  const uint32_t hb = __float_as_uint(h), lb = __float_as_uint(l);
  const uint32_t some = min(lb << 1, 1u);                     // l is not zero
  const uint32_t below = ((hb ^ lb) >> 31) & some;            // |hi + lo| < |h|
  const uint32_t b = (hb - below) | some;
  return fabsf(h) < __builtin_inff() ? __uint_as_float(b) : h;
}

// the same from 64 bits
__device__ __forceinline__ float round_odd(double y) {
  const float h = (float)y;
  return fabsf(h) < __builtin_inff() ? round_odd(h, (float)(y - (double)h)) : h;
}

template <int CTRL>
__device__ __forceinline__ double butterfly_xlane64(double own, bool upper) {
  const uint64_t b = __builtin_bit_cast(uint64_t, own);
  const uint64_t p = (uint64_t)dpp_u32<CTRL>((uint32_t)b) |
                     (uint64_t)dpp_u32<CTRL>((uint32_t)(b >> 32)) << 32;
  const double partner = __builtin_bit_cast(double, p);
  return upper ? partner - own : partner + own;
}

// random signs and the unnormalised 32-point transform of a block held by a quad, in 64 bits
__device__ __forceinline__ void hadamard_quad64(double (&w)[8], int q, uint32_t sign_mask) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if ((sign_mask >> (8 * q + k)) & 1u) w[k] = -w[k];
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i & h) continue;
      const double a = w[i], b = w[i + h];
      w[i] = a + b;
      w[i + h] = a - b;
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = butterfly_xlane64<kQuadXor1>(w[k], q & 1);
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = butterfly_xlane64<kQuadXor2>(w[k], q & 2);
}

// v of the lane across: 8 lanes (row_ror 8) and less inside a row of 16, then 16 and 32 lanes away.
// Each returns v + its partner's v.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + dpp_f32<CTRL>(v);
}
template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t p = (uint64_t)dpp_u32<CTRL>((uint32_t)b) |
                     (uint64_t)dpp_u32<CTRL>((uint32_t)(b >> 32)) << 32;
  return v + __builtin_bit_cast(double, p);
}
__device__ __forceinline__ float add_halves(float v) {
  uint32_t b = __float_as_uint(v);
  auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  b = __float_as_uint(v);
  r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ double add_halves(double v) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t l = (uint32_t)b, h = (uint32_t)(b >> 32);
    const auto rl = k ? __builtin_amdgcn_permlane32_swap(l, l, false, false)
                      : __builtin_amdgcn_permlane16_swap(l, l, false, false);
    const auto rh = k ? __builtin_amdgcn_permlane32_swap(h, h, false, false)
                      : __builtin_amdgcn_permlane16_swap(h, h, false, false);
    v = __builtin_bit_cast(double, (uint64_t)rh[0] << 32 | rl[0]) +
        __builtin_bit_cast(double, (uint64_t)rh[1] << 32 | rl[1]);
  }
  return v;
}

// Sum over the T threads of a row (16 or 64 lanes, or several waves of the workgroup, all of which
// take part); every thread gets the same value. red: one value a wave, in one of two areas in turn
// from one row to the next, so that one barrier a row is enough.
template <int T, class F>
__device__ __forceinline__ F row_sum(F v, F* red) {
  static_assert(T == 16 || T % 64 == 0);
  v = add_dpp<kRowRor8>(add_dpp<kRowRor4>(add_dpp<kQuadXor2>(add_dpp<kQuadXor1>(v))));
  if constexpr (T >= 64) v = add_halves(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    red += threadIdx.x / T * (T / 64);
    v = red[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v += red[w];
  }
  return v;
}

// 1 / sqrt(a) to about 2^-52: the hardware's approximation and one step of third order (its error
// e = 1 - a r^2 enters with e^3). Zero and infinity as the division gives them.
__device__ __forceinline__ double inv_sqrt(double a) {
  const double r = __builtin_amdgcn_rsq(a);
  const double e = fma(-a * r, r, 1.0);
  const double f = fma(r * e, fma(e, 0.375, 0.5), r);
  return a > 0.0 && a < __builtin_inf() ? f : r;
}

// a chunk of 8 values as it is in memory
template <bool BF16>
struct RawChunk {
  u32x4 w[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ RawChunk<BF16> load_raw(const void* p, int64_t off) {
  RawChunk<BF16> o;
  const u32x4* q = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(p) +
                                                  off * (BF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) o.w[i] = q[i];
  return o;
}

template <bool BF16>
__device__ __forceinline__ void store_raw(void* p, int64_t off, const RawChunk<BF16>& v) {
  u32x4* q = reinterpret_cast<u32x4*>(reinterpret_cast<uint8_t*>(p) + off * (BF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) q[i] = v.w[i];
}

template <bool BF16>
__device__ __forceinline__ void values(const RawChunk<BF16>& c, float (&v)[8]) {
  if constexpr (BF16) {
    widen_bf16x8(c.w[0], v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(c.w[k >> 2][k & 3]);
  }
}

template <bool BF16>
__device__ __forceinline__ RawChunk<BF16> raw_of(const float (&v)[8]) {
  RawChunk<BF16> o;
  if constexpr (BF16) {
    o.w[0] = pack_bf16x8(v);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o.w[i][k] = __float_as_uint(v[4 * i + k]);
  }
  return o;
}

// FMT: 0 no codes, 1 E2M1, 2 E4M3, 3 E5M2. T threads hold a row, V chunks of 8 values each. A
// workgroup walks over rows with the weights in registers, the next row's values on the way while
// one is normalised (for up to 2 chunks a thread). Loads past the row or the last row repeat valid
// places instead of branching: a wait behind a branch would have to count on none of the loads and
// stores in it.
// Bound by HBM: 16384 x 8192 bf16 with residual, y and E4M3 codes 205 to 228 us from card to card
// (5.3 to 5.9 TB/s of 9 bytes an element; 225 to 231 on one with 4 to 12 waves a SIMD), 8192 x 4096
// 59 us; rows of 128 by the vector ALU (25 to 28 us for 262144, 3.9 TB/s), as are stochastic rounding
// and the rotation: to MXFP4 without y, 8192 x 4096, 43 us nearest, 59 stochastic, 79 and 87 rotated.
template <bool BF16, int T, int V, int FMT, bool SR, bool RES>
__global__ __launch_bounds__(T > 256 ? T : 256) void rmsnorm_kernel(const NormArgs a) {
  constexpr int kThreads = T > 256 ? T : 256;
  constexpr int kRows = kThreads / T;
  constexpr bool kAhead = V < 4;  // 4 chunks leave no registers for the next row's
  __shared__ double red[2][T > 64 ? T / 64 : 1];
  const int t = threadIdx.x % T, sub = threadIdx.x / T;
  const int nch = (int)(a.cols / 8);
  float g[V][8];
  int col[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = t + v * T;
    col[v] = 8 * (c < nch ? c : nch - 1);
    load_gamma(a.gamma, a.gamma_bf16, col[v], g[v]);
  }
  const int64_t stride = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + sub;
  RawChunk<BF16> x[V], r[RES ? V : 1];
  auto load_row = [&](int64_t i) {
    i = i < a.rows ? i : a.rows - 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = load_raw<BF16>(a.x, i * a.ldx + col[v]);
      if constexpr (RES) r[v] = load_raw<BF16>(a.residual, i * a.ldr + col[v]);
    }
  };
  if constexpr (kAhead) load_row(row);
  for (int par = 0; row - sub < a.rows; row += stride, par ^= 1) {
    const bool live = row < a.rows;
    if constexpr (!kAhead) load_row(row);
    RawChunk<BF16> s[V];
    double ss = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float w[8];
      values<BF16>(x[v], w);
      s[v] = x[v];
      if constexpr (RES) {
        float q[8];
        values<BF16>(r[v], q);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] += q[k];
        s[v] = raw_of<BF16>(w);
        values<BF16>(s[v], w);  // the stored sum is what is normalised
      }
      if (t + v * T < nch) {
        if (a.sum && live) store_raw<BF16>(a.sum, row * a.lds + col[v], s[v]);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fma((double)w[k], (double)w[k], ss);
      }
    }
    if constexpr (kAhead) load_row(row + stride);
    ss = row_sum<T>(ss, red[par]);
    const double rho = inv_sqrt(fma(ss, a.inv_cols, (double)a.eps));
    if (!live) continue;
    if (a.rstd && t == 0) a.rstd[row] = (float)rho;
    // rows of extreme size: 2^64 moves from one factor of s rho to the other
    const double scale = rho < 0x1p-90 ? 0x1p64 : rho > 0x1p90 ? 0x1p-64 : 1.0;
    const float rho_hi = (float)(rho * scale), rho_lo = (float)(rho * scale - (double)rho_hi);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (t + v * T >= nch) continue;  // whole quads: cols is a multiple of 32
      float w[8], hi[8], lo[8];
      values<BF16>(s[v], w);
      if (scale != 1.0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] *= (float)(1.0 / scale);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        product(w[k], rho_hi, rho_lo, g[v][k], hi[k], lo[k]);
        w[k] = sum_of(hi[k], lo[k]);
      }
      if constexpr (SR) {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = round_odd(hi[k], lo[k]);
      } else if constexpr (BF16 || FMT != 0) {
        // The nearest fp32 value serves as well, unless it is a tie of the next rounding (or a
        // power of two that the block maximum may only just miss, or an infinity's NaN): with 8
        // significant bits at most, those have 15 zero bits at the end. One chunk in 4096.
        uint32_t low = __float_as_uint(w[0]) << 17;
#pragma unroll
        for (int k = 1; k < 8; ++k) low = min(low, __float_as_uint(w[k]) << 17);
        if (low == 0u) {
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = round_odd(hi[k], lo[k]);
        }
      }
      if (a.y) {
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = BF16 ? w[k] : nearest(hi[k], lo[k]);
        store_raw<BF16>(a.y, row * a.ldy + col[v], raw_of<BF16>(o));
      }
      if constexpr (FMT != 0) {
        if (a.hadamard) {
          double y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            y[k] = __builtin_copysign((double)hi[k] + (double)lo[k], (double)hi[k]);
          hadamard_quad64(y, t & 3, a.sign_mask);
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = round_odd(y[k]);
        }
        const int64_t at = row * nch + t + v * T;  // chunk of the codes and of the random fields
        uint32_t sb;
        if constexpr (FMT == 1) {
          const uint32_t code = a.ceil
              ? quant_chunk8<false, SR, true>(w, t & 3, 0u, a.seed, (uint64_t)at, sb)
              : quant_chunk8<false, SR, false>(w, t & 3, 0u, a.seed, (uint64_t)at, sb);
          reinterpret_cast<uint32_t*>(a.codes)[at] = code;
        } else {
          const uint2 code = a.ceil
              ? quant_chunk8_fp8<FMT - 2, false, SR, true>(w, t & 3, 0u, a.seed, (uint64_t)at, sb)
              : quant_chunk8_fp8<FMT - 2, false, SR, false>(w, t & 3, 0u, a.seed, (uint64_t)at, sb);
          reinterpret_cast<uint2*>(a.codes)[at] = code;
        }
        if ((t & 3) == 0) a.scales[at >> 2] = (uint8_t)sb;
      }
    }
  }
}

template <bool BF16, int T, int V, int FMT, bool SR>
hipError_t launch_norm(NormArgs a) {
  constexpr int kThreads = T > 256 ? T : 256;
  constexpr int kRows = kThreads / T;
  const int64_t want = (a.rows + kRows - 1) / kRows;
  const int64_t most = kNormThreads / kThreads;
  const dim3 grid((unsigned)(want < most ? want : most)), block(kThreads);
  a.inv_cols = 1.0 / (double)a.cols;
  if (a.residual)
    hipLaunchKernelGGL((rmsnorm_kernel<BF16, T, V, FMT, SR, true>), grid, block, 0,
                       (hipStream_t)a.stream, a);
  else
    hipLaunchKernelGGL((rmsnorm_kernel<BF16, T, V, FMT, SR, false>), grid, block, 0,
                       (hipStream_t)a.stream, a);
  return hipGetLastError();
}

// The shape of a row's threads by its columns: T threads, V chunks of 8 each.
template <class F>
auto with_shape(int64_t cols, F&& f) {
  using std::integral_constant;
  auto shape = [&](auto t, auto v) { return f(t, v); };
#define MX_SHAPE(T, V) return shape(integral_constant<int, T>{}, integral_constant<int, V>{})
  if (cols <= 128) MX_SHAPE(16, 1);
  if (cols <= 512) MX_SHAPE(64, 1);
  if (cols <= 1024) MX_SHAPE(64, 2);
  if (cols <= 2048) MX_SHAPE(256, 1);
  if (cols <= 4096) MX_SHAPE(256, 2);
  if (cols <= 8192) MX_SHAPE(512, 2);
  if (cols <= 16384) MX_SHAPE(1024, 2);
  MX_SHAPE(1024, 4);
#undef MX_SHAPE
}

template <bool BF16, int FMT, bool SR>
hipError_t pick_norm_shape(const NormArgs& a) {
  return with_shape(a.cols,
                    [&](auto t, auto v) { return launch_norm<BF16, t(), v(), FMT, SR>(a); });
}

template <bool BF16>
hipError_t pick_norm_format(const NormArgs& a) {
  switch (a.fmt) {
    case 0: return pick_norm_shape<BF16, 0, false>(a);
    case 1: return a.sr ? pick_norm_shape<BF16, 1, true>(a) : pick_norm_shape<BF16, 1, false>(a);
    case 2: return a.sr ? pick_norm_shape<BF16, 2, true>(a) : pick_norm_shape<BF16, 2, false>(a);
    default: return a.sr ? pick_norm_shape<BF16, 3, true>(a) : pick_norm_shape<BF16, 3, false>(a);
  }
}

// ---------------------------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------------------------
// A workgroup walks over rows like the forward kernel and keeps its columns' sums of dy z in
// registers; rmsnorm_dgamma_kernel joins the workgroups' sums, partial[block][cols], in a fixed
// order. Two rows and more a workgroup halve what it has to read.
// Bound by HBM: 16384 x 8192 bf16 with dsum 192 to 201 us (5.3 to 5.6 TB/s of 8 bytes an element),
// 8192 x 4096 50 us; the join of either 4 to 5 us more.
// SMALL (below): 512 threads also for narrow rows, for the columns' sake (4096 x 32 bf16: 6.1 us, 8.8
// with 256 threads).
template <bool BF16, int T, bool SMALL>
constexpr int kBackwardThreads =
    T <= 64 ? (SMALL ? 512 : 256) : T <= 256 || (BF16 && T <= 512) ? 2 * T : T;

// dgamma of columns 32 i .. 32 i + 31 over all rows, for tensors that the caches hold: 4 threads a
// row, every 4th lane another one.
template <bool BF16, int THREADS>
__device__ __forceinline__ void dgamma_columns(const NormBackwardArgs& a, int i) {
  __shared__ float part[THREADS / 64][32];
  const int c = threadIdx.x & 3;
  const int64_t col = 32 * (int64_t)i + 8 * c;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int64_t row = threadIdx.x >> 2; row < a.rows; row += THREADS / 4) {
    float y[8], z[8];
    values<BF16>(load_raw<BF16>(a.dy, row * a.lddy + col), y);
    values<BF16>(load_raw<BF16>(a.s, row * a.lds + col), z);
    const float r = a.rstd[row];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] += y[k] * (z[k] * r);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float v = add_halves(add_dpp<kRowRor8>(add_dpp<kRowRor4>(acc[k])));
    if ((threadIdx.x & 63) < 4) part[threadIdx.x >> 6][8 * c + k] = v;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    float v = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) v += part[w][threadIdx.x];
    a.dgamma[32 * (int64_t)i + threadIdx.x] = v;
  }
}

// SMALL: the first workgroups form dgamma from the columns, beside the rows: one launch and no
// workspace. They come first because they take longest (1024 x 4096 fp32: 16.8 us, 20.4 last).
template <bool BF16, int T, int V, bool DSUM, bool SMALL>
__global__ __launch_bounds__((kBackwardThreads<BF16, T, SMALL>)) void rmsnorm_backward_kernel(
    const NormBackwardArgs a) {
  constexpr int kThreads = kBackwardThreads<BF16, T, SMALL>;
  constexpr int kRows = kThreads / T;
  int block = (int)blockIdx.x;
  if constexpr (SMALL) {
    const int columns = a.dgamma ? (int)(a.cols / 32) : 0;
    if (block < columns) {
      dgamma_columns<BF16, kThreads>(a, block);
      return;
    }
    block -= columns;
  }
  // The widest rows leave no registers for the next row's values (16 waves have 128 each), nor for
  // their own between the sum and the result: they are read again, from the caches.
  constexpr bool kAhead = V < 4 && (BF16 || T < 1024);
  __shared__ float red[2][kThreads / 64];
  __shared__ float join[!SMALL && kRows > 1 ? kRows : 1][!SMALL && kRows > 1 ? T * V * 8 : 1];
  const int t = threadIdx.x % T, sub = threadIdx.x / T;
  const int nch = (int)(a.cols / 8);
  float g[V][8], acc[V][8];  // g only where the next row is loaded ahead
  int col[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = t + v * T;
    col[v] = 8 * (c < nch ? c : nch - 1);
    if constexpr (kAhead) load_gamma(a.gamma, a.gamma_bf16, col[v], g[v]);
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[v][k] = 0.0f;
  }
  const int64_t stride = (int64_t)a.row_blocks * kRows;
  int64_t row = (int64_t)block * kRows + sub;
  constexpr int kHeld = kAhead ? V : 1;
  RawChunk<BF16> dy[kHeld], s[kHeld], d[DSUM ? kHeld : 1];
  float rho;
  auto load_row = [&](int64_t i) {
    i = i < a.rows ? i : a.rows - 1;
    rho = a.rstd[i];
#pragma unroll
    for (int v = 0; v < kHeld; ++v) {
      dy[v] = load_raw<BF16>(a.dy, i * a.lddy + col[v]);
      s[v] = load_raw<BF16>(a.s, i * a.lds + col[v]);
    }
#pragma unroll
    for (int v = 0; v < kHeld; ++v)
      if constexpr (DSUM) d[v] = load_raw<BF16>(a.dsum, i * a.ldds + col[v]);
  };
  // a chunk's share of the sum of u z, and its dy z
  auto first = [&](int v, const RawChunk<BF16>& cy, const RawChunk<BF16>& cs, const float (&w)[8],
                   float r, bool on, float& sum) {
    float y[8], z[8];
    values<BF16>(cy, y);
    values<BF16>(cs, z);
    if (on) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float p = y[k] * (z[k] * r);  // dy z
        if constexpr (!SMALL) acc[v][k] += p;
        sum = fmaf(p, w[k], sum);
      }
    }
  };
  auto second = [&](int v, const RawChunk<BF16>& cy, const RawChunk<BF16>& cs,
                    const RawChunk<BF16>& cd, const float (&w)[8], float r, float mean) {
    float y[8], z[8], o[8];
    values<BF16>(cy, y);
    values<BF16>(cs, z);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = r * (y[k] * w[k] - z[k] * r * mean);
    if constexpr (DSUM) {
      values<BF16>(cd, y);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] += y[k];
    }
    store_raw<BF16>(a.dx, row * a.lddx + col[v], raw_of<BF16>(o));
  };
  if constexpr (kAhead) load_row(row);
  for (int par = 0; row - sub < a.rows; row += stride, par ^= 1) {
    const bool live = row < a.rows;
    float sum = 0.0f;
    if constexpr (kAhead) {
      RawChunk<BF16> y0[V], s0[V], d0[DSUM ? V : 1];
      const float r = rho;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        y0[v] = dy[v];
        s0[v] = s[v];
        if constexpr (DSUM) d0[v] = d[v];
        first(v, y0[v], s0[v], g[v], r, live && t + v * T < nch, sum);
      }
      load_row(row + stride);
      const float mean = row_sum<T>(sum, red[par]) * a.inv_cols;
      if (!live) continue;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (t + v * T < nch) second(v, y0[v], s0[v], d0[DSUM ? v : 0], g[v], r, mean);
    } else {
      const int64_t i = live ? row : a.rows - 1;
      const float r = a.rstd[i];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float w[8];
        load_gamma(a.gamma, a.gamma_bf16, col[v], w);
        first(v, load_raw<BF16>(a.dy, i * a.lddy + col[v]), load_raw<BF16>(a.s, i * a.lds + col[v]),
              w, r, live && t + v * T < nch, sum);
      }
      const float mean = row_sum<T>(sum, red[par]) * a.inv_cols;
      if (!live) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (t + v * T >= nch) continue;
        float w[8];
        load_gamma(a.gamma, a.gamma_bf16, col[v], w);
        RawChunk<BF16> cd = {};
        if constexpr (DSUM) cd = load_raw<BF16>(a.dsum, i * a.ldds + col[v]);
        second(v, load_raw<BF16>(a.dy, i * a.lddy + col[v]),
               load_raw<BF16>(a.s, i * a.lds + col[v]), cd, w, r, mean);
      }
    }
  }
  if constexpr (!SMALL) {
    if (!a.partial) return;
    float* const out = a.partial + (int64_t)blockIdx.x * a.cols;
    if constexpr (kRows > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k) join[sub][(t + v * T) * 8 + k] = acc[v][k];
      __syncthreads();
      for (int c = threadIdx.x; c < (int)a.cols; c += kThreads) {
        float p = join[0][c];
#pragma unroll
        for (int i = 1; i < kRows; ++i) p += join[i][c];
        out[c] = p;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (t + v * T < nch) store_raw<false>(out, col[v], raw_of<false>(acc[v]));
    }
  }
}

// dgamma[c] = sum of the workgroups' sums, in 64 bits: 16 columns by 64 slices of the workgroups,
// 4 columns a thread
__global__ __launch_bounds__(256) void rmsnorm_dgamma_kernel(const float* __restrict__ partial,
                                                             int blocks, int64_t cols,
                                                             float* __restrict__ dgamma) {
  __shared__ double part[64][17];
  const int c = threadIdx.x & 3, slice = threadIdx.x >> 2;
  const float* p = partial + (int64_t)blockIdx.x * 16 + 4 * c;  // cols is a multiple of 32
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 8
  for (int b = slice; b < blocks; b += 64) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(p + b * cols);
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] += (double)v[k];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) part[slice][4 * c + k] = sum[k];
  __syncthreads();
  const int col = threadIdx.x & 15, q = threadIdx.x >> 4;  // 4 slices a thread, then 16 threads
  double s = part[4 * q][col];
#pragma unroll
  for (int i = 1; i < 4; ++i) s += part[4 * q + i][col];
  __syncthreads();
  part[q][col] = s;
  __syncthreads();
  if (threadIdx.x < 16) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][col];
    dgamma[(int64_t)blockIdx.x * 16 + col] = (float)s;
  }
}

// workgroups of the backward kernel: what 256 compute units hold at 6 waves a SIMD with one chunk
// a thread, 4 with more; fewer for few rows, whose sums would be as much traffic as the rows
template <bool BF16, int T, int V>
int64_t backward_blocks(int64_t rows) {
  constexpr int kThreads = kBackwardThreads<BF16, T, false>;
  constexpr int kRows = kThreads / T;
  constexpr int64_t most = 256 * 4 * 64 * (V == 1 ? 6 : 4) / kThreads;
  const int64_t want = (rows + kRows - 1) / kRows;
  if (want <= 256) return want;
  const int64_t few = want / 4 > 256 ? want / 4 : 256;
  return few < most ? few : most;
}

// Tensors whose dgamma is formed from the columns: dy and s are read twice, the second time from
// the caches, and each of the cols / 32 workgroups walks over all rows, so their number is bounded
// as well as the tensor's size. Kernel times in us, columns | the workgroups' sums and their join
// (which costs a caller without a graph 3 us on the host besides: a second launch, a workspace):
//   777 x 2720 fp32 9.2 | 11.4     1024 x 1024 bf16 3.8 | 7.3    2048 x 128 bf16 4.4 | 5.2
//   4096 x 32 bf16 6.1 | 5.4       4096 x 128 bf16 6.3 | 6.0     4096 x 1024 bf16 21.7 | 10.4
//   8192 x 32 bf16 10.3 | 5.9      8192 x 512 bf16 36 | 11       131072 x 32 bf16 326 | 18
bool small_backward(int64_t rows, int64_t cols) {
  return rows <= 4096 && rows * cols <= (1 << 22);
}

template <bool BF16, int T, int V, bool DSUM>
hipError_t launch_backward(NormBackwardArgs a) {
  a.inv_cols = 1.0f / (float)a.cols;
  if (small_backward(a.rows, a.cols)) {
    constexpr int kThreads = kBackwardThreads<BF16, T, true>;
    a.row_blocks = (int)((a.rows + kThreads / T - 1) / (kThreads / T));
    const unsigned blocks = a.row_blocks + (a.dgamma ? (unsigned)(a.cols / 32) : 0u);
    hipLaunchKernelGGL((rmsnorm_backward_kernel<BF16, T, V, DSUM, true>), dim3(blocks),
                       dim3(kThreads), 0, (hipStream_t)a.stream, a);
    return hipGetLastError();
  }
  a.row_blocks = (int)backward_blocks<BF16, T, V>(a.rows);
  hipLaunchKernelGGL((rmsnorm_backward_kernel<BF16, T, V, DSUM, false>),
                     dim3((unsigned)a.row_blocks), dim3((kBackwardThreads<BF16, T, false>)), 0,
                     (hipStream_t)a.stream, a);
  if (hipError_t e = hipGetLastError(); e != hipSuccess || !a.dgamma) return e;
  hipLaunchKernelGGL(rmsnorm_dgamma_kernel, dim3((unsigned)(a.cols / 16)), dim3(256), 0,
                     (hipStream_t)a.stream, a.partial, a.row_blocks, a.cols, a.dgamma);
  return hipGetLastError();
}

}  // namespace

int64_t mx_norm_backward_blocks(int64_t rows, int64_t cols) {
  if (small_backward(rows, cols)) return 0;
  return with_shape(cols, [&](auto t, auto v) {
    const int64_t b = backward_blocks<true, t(), v()>(rows), f = backward_blocks<false, t(), v()>(rows);
    return b > f ? b : f;
  });
}

hipError_t mx_launch_rmsnorm(const NormArgs& a) {
  return a.bf16 ? pick_norm_format<true>(a) : pick_norm_format<false>(a);
}

hipError_t mx_launch_rmsnorm_backward(const NormBackwardArgs& a) {
  return with_shape(a.cols, [&](auto t, auto v) {
    if (a.dsum)
      return a.bf16 ? launch_backward<true, t(), v(), true>(a)
                    : launch_backward<false, t(), v(), true>(a);
    return a.bf16 ? launch_backward<true, t(), v(), false>(a)
                  : launch_backward<false, t(), v(), false>(a);
  });
}
