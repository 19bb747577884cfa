// norm.hip — RMS norm with the residual's addition and a block-scaled output, and its backward
// pass, for gfx950.
//
// Forward, per row:  s = x + r (fp32, rounded to the tensors' type: the residual stream that is
// stored is the value that is normalised, so the backward pass and a recomputation from the
// stored sum see the same numbers),  rho = 1 / sqrt(mean(s^2) + eps),  y = s rho g.
// y is formed in 64 bits and rounded once to every output's type (see odd32), so the outputs do
// not depend on the order of the sum, that is on the launch shape or on how many rows share the
// call.
// Backward:  u = dy g, z = s rho, c = mean(u z):  dx = rho (u - z c) (+ dsum),  dg = sum_rows dy z.
#include "mx_device.h"
#include "mx_launch.h"

using namespace mxd;

namespace {

constexpr int kMaxBlocks = 1 << 20;  // workgroups walk over the rows beyond this many

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

template <bool BF16>
__device__ __forceinline__ void store_chunk(void* p, int64_t off, const float (&v)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p) + off) = pack_bf16x8(v);
  } else {
    f32x4* q = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + off);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
  }
}

__device__ __forceinline__ void load_gamma(const void* g, bool bf16, int64_t off, float (&v)[8]) {
  if (bf16) load_chunk<true>(g, off, v);
  else load_chunk<false>(g, off, v);
}

// fp32 by rounding to odd: toward zero, with the last bit set when bits were dropped. A rounding
// of the result to at most 22 significant bits (bf16, E4M3, E5M2, E2M1, the thresholds of the
// stochastic rounding, the block maximum's exponent) is then the rounding of the 64-bit value
// itself: no tie is made or lost on the way. A value past fp32's range is infinite.
__device__ __forceinline__ float odd32(double y) {
  const float h = (float)y;
  const double d = (double)h;
  uint32_t b = __float_as_uint(h);
  if ((b & 0x7FFFFFFFu) < 0x7F800000u) {
    b -= fabs(d) > fabs(y) ? 1u : 0u;
    b |= d != y ? 1u : 0u;
  }
  return __uint_as_float(b);
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

// Sum over the T threads of a row (T divides 64, or the row has the whole workgroup); every
// thread gets it. red: kWaves values, alternating between two areas from one row to the next, so
// one barrier a row is enough.
template <int T, class F>
__device__ __forceinline__ F row_sum(F v, F* red) {
#pragma unroll
  for (int m = 1; m < (T < 64 ? T : 64); m <<= 1) v += __shfl_xor(v, m);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v += red[w];
  }
  return v;
}

// FMT: 0 no codes, 1 E2M1, 2 E4M3, 3 E5M2. T threads hold a row, V chunks of 8 values each.
template <bool BF16, int T, int V, int FMT, bool SR>
__global__ __launch_bounds__(T > 256 ? T : 256) void rmsnorm_kernel(const NormArgs a) {
  constexpr int kThreads = T > 256 ? T : 256;
  constexpr int kRows = kThreads / T;
  __shared__ double red[2][T > 64 ? T / 64 : 1];
  const int t = threadIdx.x % T, sub = threadIdx.x / T;
  const int nch = (int)(a.cols / 8);
  int par = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < a.rows;
       row0 += (int64_t)gridDim.x * kRows, par ^= 1) {
    const int64_t row = row0 + sub;
    const bool live = row < a.rows;
    float s[V][8];
    double ss = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * T;
      if (live && c < nch) {
        load_chunk<BF16>(a.x, row * a.ldx + 8 * c, s[v]);
        if (a.residual) {
          float r[8];
          load_chunk<BF16>(a.residual, row * a.ldr + 8 * c, r);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            s[v][k] += r[k];
            if (BF16) s[v][k] = (float)(__bf16)s[v][k];  // the stored sum is what is normalised
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) s[v][k] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fma((double)s[v][k], (double)s[v][k], ss);
    }
    ss = row_sum<T>(ss, red[par]);
    const double rho = 1.0 / sqrt(ss / (double)a.cols + (double)a.eps);
    if (!live) continue;
    if (a.rstd && t == 0) a.rstd[row] = (float)rho;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * T;
      if (c >= nch) continue;  // whole quads: cols is a multiple of 32
      if (a.sum) store_chunk<BF16>(a.sum, row * a.lds + 8 * c, s[v]);
      float g[8];
      load_gamma(a.gamma, a.gamma_bf16, 8 * c, g);
      double y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = (double)s[v][k] * rho * (double)g[k];
      if (a.y) {
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = BF16 ? odd32(y[k]) : (float)y[k];
        store_chunk<BF16>(a.y, row * a.ldy + 8 * c, o);
      }
      if constexpr (FMT != 0) {
        if (a.hadamard) hadamard_quad64(y, t & 3, a.sign_mask);
        float w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = odd32(y[k]);
        const int64_t at = row * nch + c;  // chunk index in the codes and for the random fields
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
hipError_t launch_norm(const NormArgs& a) {
  constexpr int kThreads = T > 256 ? T : 256;
  constexpr int kRows = kThreads / T;
  const int64_t want = (a.rows + kRows - 1) / kRows;
  const unsigned blocks = (unsigned)(want < kMaxBlocks ? want : kMaxBlocks);
  hipLaunchKernelGGL((rmsnorm_kernel<BF16, T, V, FMT, SR>), dim3(blocks), dim3(kThreads), 0,
                     (hipStream_t)a.stream, a);
  return hipGetLastError();
}

template <bool BF16, int FMT, bool SR>
hipError_t pick_norm_shape(const NormArgs& a) {
  if (a.cols <= 128) return launch_norm<BF16, 16, 1, FMT, SR>(a);
  if (a.cols <= 512) return launch_norm<BF16, 64, 1, FMT, SR>(a);
  if (a.cols <= 1024) return launch_norm<BF16, 64, 2, FMT, SR>(a);
  if (a.cols <= 2048) return launch_norm<BF16, 64, 4, FMT, SR>(a);
  if (a.cols <= 4096) return launch_norm<BF16, 256, 2, FMT, SR>(a);
  if (a.cols <= 8192) return launch_norm<BF16, 256, 4, FMT, SR>(a);
  if (a.cols <= 16384) return launch_norm<BF16, 1024, 2, FMT, SR>(a);
  return launch_norm<BF16, 1024, 4, FMT, SR>(a);
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
constexpr int kBwdBlocks = 1024;  // partial sums of the weight gradient

// Every workgroup walks over rows blockIdx, blockIdx + gridDim, ... and keeps its columns' sums
// of dy z in registers; partial[block][cols] are joined by rmsnorm_dgamma_kernel in a fixed order.
template <bool BF16, int T, int V>
__global__ __launch_bounds__(T > 256 ? T : 256) void rmsnorm_backward_kernel(
    const NormBackwardArgs a) {
  constexpr int kThreads = T > 256 ? T : 256;
  constexpr int kRows = kThreads / T;
  __shared__ float red[2][T > 64 ? T / 64 : 1];
  __shared__ float join[kRows > 1 ? kRows : 1][kRows > 1 ? T * V * 8 : 1];
  const int t = threadIdx.x % T, sub = threadIdx.x / T;
  const int nch = (int)(a.cols / 8);
  float g[V][8], acc[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = t + v * T;
#pragma unroll
    for (int k = 0; k < 8; ++k) g[v][k] = acc[v][k] = 0.0f;
    if (c < nch) load_gamma(a.gamma, a.gamma_bf16, 8 * c, g[v]);
  }
  const float inv_cols = 1.0f / (float)a.cols;
  int par = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < a.rows;
       row0 += (int64_t)gridDim.x * kRows, par ^= 1) {
    const int64_t row = row0 + sub;
    const bool live = row < a.rows;
    const float rho = live ? a.rstd[row] : 0.0f;
    float dy[V][8], z[V][8];
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * T;
      if (live && c < nch) {
        load_chunk<BF16>(a.dy, row * a.lddy + 8 * c, dy[v]);
        load_chunk<BF16>(a.s, row * a.lds + 8 * c, z[v]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) dy[v][k] = z[v][k] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        z[v][k] *= rho;
        acc[v][k] = fmaf(dy[v][k], z[v][k], acc[v][k]);
        sum = fmaf(dy[v][k] * g[v][k], z[v][k], sum);
      }
    }
    const float mean = row_sum<T>(sum, red[par]) * inv_cols;
    if (!live) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * T;
      if (c >= nch) continue;
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = rho * (dy[v][k] * g[v][k] - z[v][k] * mean);
      if (a.dsum) {
        float d[8];
        load_chunk<BF16>(a.dsum, row * a.ldds + 8 * c, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] += d[k];
      }
      store_chunk<BF16>(a.dx, row * a.lddx + 8 * c, o);
    }
  }
  if (!a.partial) return;
  if constexpr (kRows > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int k = 0; k < 8; ++k) join[sub][(t + v * T) * 8 + k] = acc[v][k];
    __syncthreads();
    for (int c = threadIdx.x; c < (int)a.cols; c += kThreads) {
      float p = join[0][c];
#pragma unroll
      for (int r = 1; r < kRows; ++r) p += join[r][c];
      a.partial[(int64_t)blockIdx.x * a.cols + c] = p;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = t + v * T;
      if (c < nch) store_chunk<false>(a.partial, (int64_t)blockIdx.x * a.cols + 8 * c, acc[v]);
    }
  }
}

// dgamma[c] = sum over the blocks' partial sums: 32 columns by 8 slices of the blocks a workgroup
__global__ __launch_bounds__(256) void rmsnorm_dgamma_kernel(const float* __restrict__ partial,
                                                             int blocks, int64_t cols,
                                                             float* __restrict__ dgamma) {
  __shared__ double part[8][32];
  const int c = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c;  // cols is a multiple of 32
  double sum = 0.0;
  for (int b = slice; b < blocks; b += 8) sum += (double)partial[b * cols + col];
  part[slice][c] = sum;
  __syncthreads();
  if (slice == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += part[i][c];
    dgamma[col] = (float)sum;
  }
}

template <bool BF16, int T, int V>
hipError_t launch_backward(const NormBackwardArgs& a) {
  constexpr int kThreads = T > 256 ? T : 256;
  const int blocks = (int)mx_norm_backward_blocks(a.rows, a.cols);
  if (blocks > 0) {
    hipLaunchKernelGGL((rmsnorm_backward_kernel<BF16, T, V>), dim3((unsigned)blocks),
                       dim3(kThreads), 0, (hipStream_t)a.stream, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!a.dgamma) return hipSuccess;
  hipLaunchKernelGGL(rmsnorm_dgamma_kernel, dim3((unsigned)(a.cols / 32)), dim3(256), 0,
                     (hipStream_t)a.stream, a.partial, blocks, a.cols, a.dgamma);
  return hipGetLastError();
}

template <bool BF16>
hipError_t pick_backward_shape(const NormBackwardArgs& a) {
  if (a.cols <= 128) return launch_backward<BF16, 16, 1>(a);
  if (a.cols <= 512) return launch_backward<BF16, 64, 1>(a);
  if (a.cols <= 1024) return launch_backward<BF16, 64, 2>(a);
  if (a.cols <= 2048) return launch_backward<BF16, 64, 4>(a);
  if (a.cols <= 4096) return launch_backward<BF16, 256, 2>(a);
  if (a.cols <= 8192) return launch_backward<BF16, 256, 4>(a);
  if (a.cols <= 16384) return launch_backward<BF16, 1024, 2>(a);
  return launch_backward<BF16, 1024, 4>(a);
}

}  // namespace

int64_t mx_norm_backward_blocks(int64_t rows, int64_t cols) {
  const int64_t per = cols <= 128 ? 16 : cols <= 2048 ? 4 : 1;  // rows a workgroup holds at once
  const int64_t want = (rows + per - 1) / per;
  return want < kBwdBlocks ? want : kBwdBlocks;
}

hipError_t mx_launch_rmsnorm(const NormArgs& a) {
  return a.bf16 ? pick_norm_format<true>(a) : pick_norm_format<false>(a);
}

hipError_t mx_launch_rmsnorm_backward(const NormBackwardArgs& a) {
  return a.bf16 ? pick_backward_shape<true>(a) : pick_backward_shape<false>(a);
}
