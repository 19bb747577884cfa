// gemv.hip — product of a few tokens' activations (bf16 or fp32, not quantized) with MXFP4
// weights, for gfx950:  y[t][n] = 2^alpha sum_k x'[t][k] E2M1(wq[n][k]) 2^(ws[n / g][k / 32] - 127),
// x' = x, or each 32-block of x rotated by the signs and the 32-point transform when the weights
// were quantized that way.
//
// The weights are read once and are the traffic: 17/32 byte each. A wave takes 16 weight rows and
// 128 columns of K a step: lane (n, g) = (lane & 15, lane >> 4) reads the 16 code bytes of row n's
// block 4 step + g (64 contiguous bytes a row) and its scale byte, and the converter turns them
// into 32 bf16 values, exact because the scale is a power of two. v_mfma_f32_16x16x32_bf16 number
// j of the step takes values 8j .. 8j+7 of every lane as the reduction index, and the same values
// of x: the order of k inside a product is free as long as both operands share it.
//
// fp32 activations (and rotated ones) go in as three bf16 terms that add up to the fp32 value:
// x = hi + mid + lo by truncation, 8 significant bits each.
#include "mx_device.h"
#include "mx_launch.h"

using namespace mxd;

namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8;  // share a workgroup's rows, each a part of K

// 8 codes (a word) times the block's scale as 8 bf16 values
__device__ __forceinline__ bf16x8_t weights8(uint32_t w, float scale) {
  u32x4 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return __builtin_bit_cast(bf16x8_t, o);
}

// 2^(b - 127) with b = 0 the subnormal 2^-127 and b = 255 an infinity, which the converter takes
// as E8M0's NaN
__device__ __forceinline__ float e8m0(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : b << 23);
}

// v = hi + mid + lo exactly (down to bf16's least subnormal); an infinity or NaN stays in hi
__device__ __forceinline__ void split3(float v, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const uint32_t b = __float_as_uint(v);
  hi = b >> 16;
  if ((b & 0x7F800000u) == 0x7F800000u) {
    hi |= (b & 0x7FFFFFu) ? 0x40u : 0u;  // a NaN whose payload sits in the dropped bits
    mid = lo = 0u;
    return;
  }
  const float r = v - __uint_as_float(b & 0xFFFF0000u);
  const uint32_t rb = __float_as_uint(r);
  mid = rb >> 16;
  lo = __float_as_uint(r - __uint_as_float(rb & 0xFFFF0000u)) >> 16;
}

// A lane's 32 values of x for one step: row m, block b (64 or 128 bytes). SPLIT: three terms.
template <bool SPLIT>
struct Activations {
  u32x4 f[SPLIT ? 3 : 1][4];
};

template <bool BF16, bool HAD>
__device__ __forceinline__ void load_x(Activations<!BF16 || HAD>& o, const void* x, int64_t at,
                                       bool on, uint32_t sign_mask) {
  constexpr bool kSplit = !BF16 || HAD;
  if (!on) {
#pragma unroll
    for (int s = 0; s < (kSplit ? 3 : 1); ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) o.f[s][j] = u32x4{0u, 0u, 0u, 0u};
    return;
  }
  if constexpr (!kSplit) {
    const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(x) + at);
#pragma unroll
    for (int j = 0; j < 4; ++j) o.f[0][j] = p[j];
  } else {
    float v[32];
    if constexpr (BF16) {
      const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(x) + at);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float w[8];
        widen_bf16x8(p[j], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[8 * j + k] = w[k];
      }
    } else {
      const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(x) + at);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const f32x4 w = p[j];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * j + k] = w[k];
      }
    }
    if constexpr (HAD) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        v[k] = __uint_as_float(__float_as_uint(v[k]) ^ (((sign_mask >> k) & 1u) << 31));
      hadamard32_inlane(v);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h[4], m[4], l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h0, m0, l0, h1, m1, l1;
        split3(v[8 * j + 2 * i], h0, m0, l0);
        split3(v[8 * j + 2 * i + 1], h1, m1, l1);
        h[i] = h0 | h1 << 16;
        m[i] = m0 | m1 << 16;
        l[i] = l0 | l1 << 16;
      }
      o.f[0][j] = u32x4{h[0], h[1], h[2], h[3]};
      o.f[1][j] = u32x4{m[0], m[1], m[2], m[3]};
      o.f[2][j] = u32x4{l[0], l[1], l[2], l[3]};
    }
  }
}

// MT tiles of 16 tokens by RT tiles of 16 weight rows a workgroup; the waves take every kWaves-th
// step of 128 columns and their sums are joined through LDS in a fixed order.
template <bool BF16, bool HAD, int MT, int RT>
__global__ __launch_bounds__(64 * kWaves) void gemv_kernel(const GemvArgs a) {
  constexpr bool kSplit = !BF16 || HAD;
  __shared__ float red[kWaves][MT * RT * 4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const int64_t nb = a.K / 32;

  const uint8_t* wrow[RT];
  const uint8_t* srow[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int64_t n = n0 + 16 * r + i16;
    n = n < a.N ? n : a.N - 1;  // rows past the end repeat the last one and are not stored
    wrow[r] = a.w + n * (a.K / 2);
    srow[r] = a.ws + n / a.gw * nb;
  }
  f32x4 acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[m][r] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int64_t b0 = 4 * wave; b0 < nb; b0 += 4 * kWaves) {
    const int64_t b = b0 + g;
    const bool in = b < nb;
    bf16x8_t w[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      u32x4 q = {0u, 0u, 0u, 0u};
      uint32_t sb = 127u;
      if (in) {
        q = *reinterpret_cast<const u32x4*>(wrow[r] + 16 * b);
        sb = srow[r][b];
      }
      const float scale = e8m0(sb);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[r][j] = weights8(q[j], scale);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t t = m0 + 16 * m + i16;
      Activations<kSplit> x;
      load_x<BF16, HAD>(x, a.x, t * a.ldx + 32 * b, in && t < a.T, a.sign_mask);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        // the 128 products of a step are summed apart from the running sum: the matrix core
        // drops what lies 24 bits below the largest term of a sum, so short sums lose less
        f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = (kSplit ? 2 : 0); s >= 0; --s)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x.f[s][j]),
                                                        w[r][j], p, 0, 0, 0);
        acc[m][r] += p;
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][(m * RT + r) * 4 + i][lane] = acc[m][r][i];
  __syncthreads();
  const float alpha = __uint_as_float((uint32_t)(a.alpha + 127) << 23);
  for (int e = threadIdx.x; e < MT * RT * 4 * 64; e += 64 * kWaves) {
    const int slot = e >> 6, l = e & 63;
    float v = red[0][slot][l];
#pragma unroll
    for (int s = 1; s < kWaves; ++s) v += red[s][slot][l];
    v *= alpha;
    const int i = slot & 3, r = (slot >> 2) % RT, m = (slot >> 2) / RT;
    const int64_t t = m0 + 16 * m + 4 * (l >> 4) + i, n = n0 + 16 * r + (l & 15);
    if (t < a.T && n < a.N) {
      if (a.out_bf16) reinterpret_cast<__bf16*>(a.y)[t * a.ldy + n] = (__bf16)v;
      else reinterpret_cast<float*>(a.y)[t * a.ldy + n] = v;
    }
  }
}

__global__ __launch_bounds__(256) void gemv_zero_kernel(const GemvArgs a) {
  const int64_t count = a.T * a.N;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < count;
       e += (int64_t)gridDim.x * 256) {
    const int64_t at = e / a.N * a.ldy + e % a.N;
    if (a.out_bf16) reinterpret_cast<__bf16*>(a.y)[at] = (__bf16)0.0f;
    else reinterpret_cast<float*>(a.y)[at] = 0.0f;
  }
}

template <bool BF16, bool HAD, int MT, int RT>
hipError_t launch_gemv(const GemvArgs& a) {
  const int64_t gx = (a.N + 16 * RT - 1) / (16 * RT), gy = (a.T + 16 * MT - 1) / (16 * MT);
  if (gx > (1 << 22) || gy > 65535) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gemv_kernel<BF16, HAD, MT, RT>), dim3((unsigned)gx, (unsigned)gy),
                     dim3(64 * kWaves), 0, (hipStream_t)a.stream, a);
  return hipGetLastError();
}

template <bool BF16, bool HAD>
hipError_t pick_gemv(const GemvArgs& a) {
  return launch_gemv<BF16, HAD, 1, 1>(a);
}

}  // namespace

hipError_t mx_launch_gemv(const GemvArgs& a) {
  if (a.K == 0) {
    const int64_t blocks = (a.T * a.N + 255) / 256;
    hipLaunchKernelGGL(gemv_zero_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256),
                       0, (hipStream_t)a.stream, a);
    return hipGetLastError();
  }
  if (a.bf16) return a.hadamard ? pick_gemv<true, true>(a) : pick_gemv<true, false>(a);
  return a.hadamard ? pick_gemv<false, true>(a) : pick_gemv<false, false>(a);
}
