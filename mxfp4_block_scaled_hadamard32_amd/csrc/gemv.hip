// gemv.hip — product of a few tokens' activations (bf16 or fp32, not quantized) with MXFP4
// weights, for gfx950:  y[t][n] = 2^alpha sum_k x'[t][k] E2M1(wq[n][k]) 2^(ws[n / g][k / 32] - 127),
// x' = x, or each 32-block of x rotated by the signs and the 32-point transform when the weights
// were quantized that way.
//
// The weights are read once and are the traffic: 17/32 byte each. A wave takes 16 weight rows and
// 128 columns of K a step: lane (n, g) = (lane & 15, lane >> 4) reads the 16 code bytes of row n's
// block 4 step + g (64 contiguous bytes a row), and the converter turns them into 32 bf16 values,
// exact because the block's scale is a power of two. v_mfma_f32_16x16x32_bf16 number j of the step
// takes values 8j .. 8j+7 of every lane's block as its reduction index, and the same values of x:
// the order of k inside a product is free as long as both operands share it.
//
// fp32 activations (and rotated ones) go in as bf16 terms that add up to the fp32 value.
#include "mx_device.h"
#include "mx_launch.h"

#include <type_traits>

using namespace mxd;

namespace {

// the 32 weights of a block (16 code bytes), times the block's scale: byte b is 2^(b - 127), byte 0
// the subnormal 2^-127; byte 255 is an infinity here, which the converter takes as E8M0's NaN
__device__ __forceinline__ void weights_of(u32x4 q, uint32_t scale, bf16x8_t (&w)[4]) {
  const uint32_t b = scale << 23;
  const float f = __uint_as_float(b > 0x00400000u ? b : 0x00400000u);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x4 o = {
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[j], f, 0)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[j], f, 1)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[j], f, 2)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[j], f, 3))};
    w[j] = __builtin_bit_cast(bf16x8_t, o);
  }
}

// 16 bytes at any address
__device__ __forceinline__ u32x4 load16_any(const uint8_t* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// a block's 32 values of x as they are in memory
template <bool BF16>
struct RawX {
  u32x4 w[BF16 ? 4 : 8];
};

template <bool BF16>
__device__ __forceinline__ void load_x(RawX<BF16>& o, const uint8_t* p) {
#pragma unroll
  for (int j = 0; j < (BF16 ? 4 : 8); ++j) o.w[j] = reinterpret_cast<const u32x4*>(p)[j];
}

// the block's values, rotated (HAD), as NT terms of 4 x 8 bf16 values
template <bool BF16, bool HAD, int NT>
__device__ __forceinline__ void terms_of(const RawX<BF16>& x, uint32_t sign_mask,
                                         u32x4 (&f)[NT][4]) {
  if constexpr (BF16 && !HAD) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[0][j] = x.w[j];
  } else {
    float v[32];
    if constexpr (BF16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float w[8];
        widen_bf16x8(x.w[j], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[8 * j + k] = w[k];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * j + k] = __uint_as_float(x.w[j][k]);
    }
    if constexpr (HAD) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        v[k] = __uint_as_float(__float_as_uint(v[k]) ^ (((sign_mask >> k) & 1u) << 31));
      hadamard32_inlane(v);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t o[4][NT];
#pragma unroll
      for (int i = 0; i < 4; ++i) split_pair<NT>(v[8 * j + 2 * i], v[8 * j + 2 * i + 1], o[i]);
#pragma unroll
      for (int s = 0; s < NT; ++s) f[s][j] = u32x4{o[0][s], o[1][s], o[2][s], o[3][s]};
    }
  }
}

// The same with half a block a lane: values 16h .. 16h+15 in the lanes of parity h, which exchange
// them for the transform's last stage.
template <bool BF16>
struct RawHalf {
  u32x4 w[BF16 ? 2 : 4];
};

template <bool BF16, bool HAD, int NT>
__device__ __forceinline__ void half_terms_of(const RawHalf<BF16>& x, uint32_t sign_mask,
                                              u32x4 (&f)[NT][2]) {
  const int h = threadIdx.x & 1;
  float v[16];
  if constexpr (BF16) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float w[8];
      widen_bf16x8(x.w[j], w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[8 * j + k] = w[k];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[4 * j + k] = __uint_as_float(x.w[j][k]);
  }
  if constexpr (HAD) {
    const uint32_t mask = sign_mask >> (16 * h);
#pragma unroll
    for (int k = 0; k < 16; ++k)
      v[k] = __uint_as_float(__float_as_uint(v[k]) ^ (((mask >> k) & 1u) << 31));
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i & s) continue;
        const float a = v[i], c = v[i + s];
        v[i] = a + c;
        v[i + s] = a - c;
      }
    }
    const uint32_t upper = h ? 0x80000000u : 0u;
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = butterfly_xlane<kQuadXor1>(v[k], upper);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t o[4][NT];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_pair<NT>(v[8 * j + 2 * i], v[8 * j + 2 * i + 1], o[i]);
#pragma unroll
    for (int s = 0; s < NT; ++s) f[s][j] = u32x4{o[0][s], o[1][s], o[2][s], o[3][s]};
  }
}

__device__ __forceinline__ void store_y(const GemvArgs& a, int64_t at, float v) {
  v *= __uint_as_float((uint32_t)(a.alpha + 127) << 23);
  if (a.out_bf16) reinterpret_cast<__bf16*>(a.y)[at] = (__bf16)v;
  else reinterpret_cast<float*>(a.y)[at] = v;
}

// bytes between the scale rows of a segment of `seg` blocks in LDS
__host__ __device__ constexpr int scale_pitch(int seg) { return (seg + 15) / 16 * 16 + 4; }

// One token, or a few whose activations fit in LDS: RT tiles of 16 weight rows a workgroup of WV waves,
// which take turns at groups of 16 blocks of K (4 steps: 256 contiguous code bytes a row). The
// workgroup first brings the activations (rotated and split there, once) and its rows' scale bytes
// into LDS, so the loop's only requests to memory are the codes: a step's registers are loaded
// with the same step of the wave's next group as soon as they have been used. A segment of K
// (seg blocks) at a time when LDS does not hold all of it. The waves' sums are joined through LDS
// in a fixed order.
template <bool BF16, bool HAD, int NT, int RT, int WV, bool ONE>
__global__ __launch_bounds__(64 * WV) void gemv_kernel(const GemvArgs a, int seg) {
  constexpr int kThreads = 64 * WV;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int T = ONE ? 1 : (int)a.T;  // a single token's addresses in LDS are constants
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);
  const int nb = (int)(a.K / 32);
  const int pitch = scale_pitch(seg);
  u32x4* const xl = reinterpret_cast<u32x4*>(lds);  // [NT][seg][4][T] pieces of 8 values
  uint8_t* const sl = lds + (size_t)NT * seg * 64 * T;
  const int64_t s0 = n0 / a.gw;  // first scale row
  const int64_t nlast = (n0 + 16 * RT < a.N ? n0 + 16 * RT : a.N) - 1;
  const int srows = (int)(nlast / a.gw - s0) + 1;

  // rows and tokens past the end repeat the last one: their products are not stored
  const uint8_t* wrow[RT];
  int soff[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int64_t n = n0 + 16 * r + i16;
    n = n < a.N ? n : a.N - 1;
    wrow[r] = a.w + n * (a.K / 2) + 16 * g;
    soff[r] = (int)(n / a.gw - s0) * pitch + g;
  }
  const int t16 = i16 < T ? i16 : T - 1;
  f32x4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int k0 = 0; k0 < nb; k0 += seg) {
    const int n = nb - k0 < seg ? nb - k0 : seg;  // blocks of this segment
    const int n4 = (n + 3) / 4 * 4, n16 = (n + 15) / 16;
    const int ng = n / 16;
    u32x4 q[4][RT];
    auto load_codes = [&](int grp, int d) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
        q[d][r] = *reinterpret_cast<const u32x4*>(wrow[r] + (int64_t)k0 * 16 + grp * 256 + 64 * d);
    };
    if (wave < ng) {
#pragma unroll
      for (int d = 0; d < 4; ++d) load_codes(wave, d);
    }
    if (k0) __syncthreads();  // the segment before has been read
    // scale bytes, then activations (zeros up to a multiple of 4 blocks)
    for (int i = threadIdx.x; i < srows * n16; i += kThreads) {
      const int row = i / n16, b = i % n16 * 16;
      const uint8_t* p = a.ws + (s0 + row) * nb + k0 + b;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (b + 16 <= n) {
        v = load16_any(p);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (b + k < n) v[k >> 2] |= (uint32_t)p[k] << (8 * (k & 3));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) *reinterpret_cast<uint32_t*>(sl + row * pitch + b + 4 * k) = v[k];
    }
    const uint8_t* const x = reinterpret_cast<const uint8_t*>(a.x);
    if constexpr (BF16 && !HAD) {
#pragma unroll 4
      for (int i = threadIdx.x; i < 4 * n4 * T; i += kThreads) {
        const int t = i / (4 * n4), p = i % (4 * n4);
        u32x4 w = {0u, 0u, 0u, 0u};
        if (p < 4 * n)
          w = *reinterpret_cast<const u32x4*>(x + (t * a.ldx + 32 * (int64_t)k0) * 2 + 16 * p);
        xl[p * T + t] = w;
      }
    } else {
      for (int i = threadIdx.x; i < n4 * T; i += kThreads) {
        const int t = i / n4, b = i % n4;
        RawX<BF16> raw = {};
        if (b < n) load_x<BF16>(raw, x + (t * a.ldx + 32 * (int64_t)(k0 + b)) * (BF16 ? 2 : 4));
        u32x4 f[NT][4];
        terms_of<BF16, HAD, NT>(raw, a.sign_mask, f);
#pragma unroll
        for (int s = 0; s < NT; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) xl[((s * seg + b) * 4 + j) * T + t] = f[s][j];
      }
    }
    __syncthreads();

    // the step of blocks b0 .. b0 + 3
    auto step = [&](const bf16x8_t (&w)[RT][4], int b0) {
      // the 128 products of a step are summed apart from the running sum: the matrix core
      // drops what lies 24 bits below the largest term of a sum, so short sums lose less
      f32x4 p[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) p[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = NT - 1; s >= 0; --s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8_t f =
              __builtin_bit_cast(bf16x8_t, xl[((s * seg + b0 + g) * 4 + j) * T + t16]);
#pragma unroll
          for (int r = 0; r < RT; ++r)
            p[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, w[r][j], p[r], 0, 0, 0);
        }
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] += p[r];
    };
    if (wave < ng) {
      int grp = wave;
      auto group = [&](auto more) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          bf16x8_t w[RT][4];
#pragma unroll
          for (int r = 0; r < RT; ++r) weights_of(q[d][r], sl[soff[r] + 16 * grp + 4 * d], w[r]);
          if constexpr (more()) load_codes(grp + WV, d);
          step(w, 16 * grp + 4 * d);
        }
        grp += WV;
      };
      while (grp + WV < ng) group(std::true_type{});
      group(std::false_type{});
    }
    for (int b0 = 16 * ng; b0 < n; b0 += 4) {
      if ((b0 / 4 + ng) % WV != wave) continue;
      bf16x8_t w[RT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        u32x4 c = {0u, 0u, 0u, 0u};  // past the end: zero codes, scale bytes and activations
        if (b0 + g < n) c = *reinterpret_cast<const u32x4*>(wrow[r] + (int64_t)(k0 + b0) * 16);
        weights_of(c, sl[soff[r] + b0], w[r]);
      }
      step(w, b0);
    }
  }

  __syncthreads();
  float* const red = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[(wave * RT * 4 + r * 4 + i) * 64 + lane] = acc[r][i];
  __syncthreads();
  for (int e = threadIdx.x; e < 16 * RT * T; e += kThreads) {
    const int t = e / (16 * RT), c = e % (16 * RT);  // token, row of the tile
    if (n0 + c >= a.N) continue;
    const float* p = red + ((c >> 4) * 4 + (t & 3)) * 64 + (t >> 2) * 16 + (c & 15);
    float v = p[0];
#pragma unroll
    for (int s = 1; s < WV; ++s) v += p[s * RT * 256];
    store_y(a, t * a.ldy + n0 + c, v);
  }
}

// Few rows or a short K: 16 tokens by RT tiles of 16 weight rows a workgroup of 8 waves, which take
// turns at groups of 16 blocks of K (16 scale bytes a row) and read the activations of their steps
// themselves. The registers of a step's codes and activations are loaded with the same step of the
// wave's next group as soon as they have been used, so 4 steps are always on the way.
template <bool BF16, bool HAD, int NT, int RT>
__global__ __launch_bounds__(512) void gemv_direct_kernel(const GemvArgs a) {
  constexpr int WV = 8;
  __shared__ float red[WV][RT * 4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  const int nb = (int)(a.K / 32);
  constexpr int kBlock = BF16 ? 64 : 128;  // bytes of a block of x

  // Rows and tokens past the end repeat the last one: their products are not stored, and no load
  // depends on a branch, which would make the waits for the loads after it count on none of them.
  const uint8_t* wrow[RT];
  const uint8_t* srow[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int64_t n = n0 + 16 * r + i16;
    n = n < a.N ? n : a.N - 1;
    wrow[r] = a.w + n * (a.K / 2) + 16 * g;
    srow[r] = a.ws + n / a.gw * nb;
  }
  const int64_t t16 = m0 + i16 < a.T ? m0 + i16 : a.T - 1;
  const uint8_t* const xrow =
      reinterpret_cast<const uint8_t*>(a.x) + t16 * a.ldx * (BF16 ? 2 : 4) + g * kBlock;
  f32x4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto load_codes = [&](u32x4 (&q)[RT], int grp, int d) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
      q[r] = *reinterpret_cast<const u32x4*>(wrow[r] + (int64_t)grp * 256 + 64 * d);
  };
  auto load_scales = [&](u32x4 (&sc)[RT], int grp) {
#pragma unroll
    for (int r = 0; r < RT; ++r) sc[r] = load16_any(srow[r] + 16 * grp);
  };
  auto multiply = [&](const bf16x8_t (&w)[RT][4], const RawX<BF16>& x) {
    u32x4 f[NT][4];
    terms_of<BF16, HAD, NT>(x, a.sign_mask, f);
    f32x4 p[RT];  // a step's products apart from the running sum, as in gemv_kernel
#pragma unroll
    for (int r = 0; r < RT; ++r) p[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = NT - 1; s >= 0; --s)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < RT; ++r)
          p[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f[s][j]),
                                                         w[r][j], p[r], 0, 0, 0);
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] += p[r];
  };

  const int ng = nb / 16;
  if (wave < ng) {
    u32x4 q[4][RT], sc[RT];
    RawX<BF16> x[4];
    int grp = wave;
    // in the order of the loop, which the waits in it count on
    load_scales(sc, grp);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      load_codes(q[d], grp, d);
      load_x<BF16>(x[d], xrow + (int64_t)(16 * grp + 4 * d) * kBlock);
    }
    auto group = [&](auto more) {
      u32x4 scn[RT];
      const int next = grp + WV;  // used if there is one
      if constexpr (more()) load_scales(scn, next);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        bf16x8_t w[RT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r) weights_of(q[d][r], (sc[r][d] >> (8 * g)) & 0xFFu, w[r]);
        if constexpr (more()) load_codes(q[d], next, d);
        multiply(w, x[d]);
        if constexpr (more()) load_x<BF16>(x[d], xrow + (int64_t)(16 * next + 4 * d) * kBlock);
      }
      if constexpr (more()) {
#pragma unroll
        for (int r = 0; r < RT; ++r) sc[r] = scn[r];
      }
      grp = next;
    };
    while (grp + WV < ng) group(std::true_type{});
    group(std::false_type{});
  }
  for (int b0 = 16 * ng; b0 < nb; b0 += 4) {
    if ((b0 / 4 + ng) % WV != wave) continue;
    const bool in = b0 + g < nb;  // past the end: zero weights and zero activations
    bf16x8_t w[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      u32x4 q = {0u, 0u, 0u, 0u};
      uint32_t sb = 0u;
      if (in) {
        q = *reinterpret_cast<const u32x4*>(wrow[r] + (int64_t)b0 * 16);
        sb = srow[r][b0 + g];
      }
      weights_of(q, sb, w[r]);
    }
    RawX<BF16> x = {};
    if (in) load_x<BF16>(x, xrow + (int64_t)b0 * kBlock);
    multiply(w, x);
  }

#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][r * 4 + i][lane] = acc[r][i];
  __syncthreads();
  for (int e = threadIdx.x; e < RT * 4 * 64; e += 64 * WV) {
    const int slot = e >> 6, l = e & 63;
    float v = red[0][slot][l];
#pragma unroll
    for (int s = 1; s < WV; ++s) v += red[s][slot][l];
    const int i = slot & 3, r = slot >> 2;
    const int64_t t = m0 + 4 * (l >> 4) + i, n = n0 + 16 * r + (l & 15);
    if (t < a.T && n < a.N) store_y(a, t * a.ldy + n, v);
  }
}

// Batches of tokens: 8 waves of RT tiles of 16 weight rows each share MT tiles of 16 tokens, which
// pass through LDS a chunk of 16 blocks of K at a time (rotated and split on the way, once a
// workgroup) while the chunk before is multiplied. A value of x is fetched once for 128 RT weight
// rows: the caches give a compute unit about 55 bytes a ns, and the codes alone want 23 of them.
// A wave's codes are requested 4 steps ahead and stay on the way across the barriers, which wait
// for LDS alone. K is cut into `splits` parts (blockIdx.z) so that few rows fill the machine too;
// their sums go to part[split][T][N] and gemv_join_kernel adds them in order.
template <bool BF16, bool HAD, int NT, int MT, int RT>
__global__ __launch_bounds__(512) void gemv_shared_kernel(const GemvArgs a, float* part,
                                                          int splits) {
  constexpr bool CONV = !BF16 || HAD;
  constexpr int kBlock = BF16 ? 64 : 128;                      // bytes of a block of x
  constexpr int kPer = CONV ? MT : 2 * MT;  // half blocks, or 16-byte pieces, of a thread
  constexpr int kBuf = NT * MT * 16 * 4 * 16;                  // 16-byte pieces of a chunk
  __shared__ u32x4 xl[2][kBuf];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, g = lane >> 4;
  const int64_t n0 = ((int64_t)blockIdx.x * 8 + wave) * (16 * RT);
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const int nb = (int)(a.K / 32);
  const int c0 = (int)((int64_t)(nb / 16) * blockIdx.z / splits);
  const int c1 = (int)((int64_t)(nb / 16) * (blockIdx.z + 1) / splits);

  // rows and tokens past the end repeat the last one: their products are not stored
  const uint8_t* wrow[RT];
  const uint8_t* srow[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int64_t n = n0 + 16 * r + i16;
    n = n < a.N ? n : a.N - 1;
    wrow[r] = a.w + n * (a.K / 2) + 16 * g;
    srow[r] = a.ws + n / a.gw * nb;
  }
  auto token = [&](int t) {
    int64_t i = m0 + t;
    i = i < a.T ? i : a.T - 1;
    return reinterpret_cast<const uint8_t*>(a.x) + i * a.ldx * (BF16 ? 2 : 4);
  };
  const uint8_t* xp[kPer];
  RawHalf<BF16> xr[CONV ? kPer : 1];
  u32x4 xc[CONV ? 1 : kPer];
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int i = threadIdx.x + 512 * p;
    if constexpr (CONV) xp[p] = token(i / 32) + i % 32 * (kBlock / 2);
    else xp[p] = token(i / 64) + i % 64 * 16;
  }
  auto fetch = [&](int c) {
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const uint8_t* q = xp[p] + (int64_t)c * 16 * kBlock;
      if constexpr (CONV) {
#pragma unroll
        for (int j = 0; j < (BF16 ? 2 : 4); ++j) xr[p].w[j] = reinterpret_cast<const u32x4*>(q)[j];
      } else {
        xc[p] = *reinterpret_cast<const u32x4*>(q);
      }
    }
  };
  // Piece (term, token tile, block, j, token) at slot token ^ (4 (block / 2) + j) % 16 of its 16:
  // the writers (neighbouring pieces of one token) spread over the banks, and the readers (16
  // tokens of blocks g, of which a 16-byte read serves tokens 0-3 and 12-15 of one block together
  // with 4-11 of its neighbour) meet no conflict: neighbours share the exchange.
  auto slot = [&](int s, int m, int b, int j, int t) {
    return (((s * MT + m) * 16 + b) * 4 + j) * 16 + (t ^ ((4 * (b >> 1) + j) & 15));
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int i = threadIdx.x + 512 * p;
      if constexpr (CONV) {
        const int t = i / 32, b = i % 32 / 2, h = i & 1;
        u32x4 f[NT][2];
        half_terms_of<BF16, HAD, NT>(xr[p], a.sign_mask, f);
#pragma unroll
        for (int s = 0; s < NT; ++s)
#pragma unroll
          for (int j = 0; j < 2; ++j) xl[buf][slot(s, t / 16, b, 2 * h + j, t & 15)] = f[s][j];
      } else {
        const int t = i / 64, q = i % 64;
        xl[buf][slot(0, t / 16, q / 4, q % 4, t & 15)] = xc[p];
      }
    }
  };
  auto sync = [] { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

  f32x4 acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[m][r] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 q[4][RT], sc[RT], scn[RT];
  auto load_codes = [&](int c, int d) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
      q[d][r] = *reinterpret_cast<const u32x4*>(wrow[r] + (int64_t)c * 256 + 64 * d);
  };
  auto load_scales = [&](u32x4 (&o)[RT], int c) {
#pragma unroll
    for (int r = 0; r < RT; ++r) o[r] = load16_any(srow[r] + 16 * c);
  };
  auto chunk = [&](int c, int buf, auto more) {
    if constexpr (more()) {
      fetch(c + 1);
      load_scales(scn, c + 1);
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      bf16x8_t w[RT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r) weights_of(q[d][r], (sc[r][d] >> (8 * g)) & 0xFFu, w[r]);
      if constexpr (more()) load_codes(c + 1, d);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 p[RT];  // a step's products apart from the running sum, as in gemv_kernel
#pragma unroll
        for (int r = 0; r < RT; ++r) p[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = NT - 1; s >= 0; --s)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8_t f =
                __builtin_bit_cast(bf16x8_t, xl[buf][slot(s, m, 4 * d + g, j, i16)]);
#pragma unroll
            for (int r = 0; r < RT; ++r)
              p[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, w[r][j], p[r], 0, 0, 0);
          }
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[m][r] += p[r];
      }
    }
    if constexpr (more()) {
      put(buf ^ 1);
#pragma unroll
      for (int r = 0; r < RT; ++r) sc[r] = scn[r];
      sync();
    }
  };
  if (c0 < c1) {
    fetch(c0);
    load_scales(sc, c0);
#pragma unroll
    for (int d = 0; d < 4; ++d) load_codes(c0, d);
    put(0);
    sync();
    int c = c0;
    for (; c + 1 < c1; ++c) chunk(c, (c - c0) & 1, std::true_type{});
    chunk(c, (c - c0) & 1, std::false_type{});
  }
  // the blocks after the last whole chunk: every wave reads its steps' activations itself
  if (blockIdx.z + 1 == (unsigned)splits) {
    for (int b0 = nb / 16 * 16; b0 < nb; b0 += 4) {
      const bool in = b0 + g < nb;  // past the end: zero weights and zero activations
      bf16x8_t w[RT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        u32x4 v = {0u, 0u, 0u, 0u};
        uint32_t s = 0u;
        if (in) {
          v = *reinterpret_cast<const u32x4*>(wrow[r] + (int64_t)b0 * 16);
          s = srow[r][b0 + g];
        }
        weights_of(v, s, w[r]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        RawX<BF16> x = {};
        if (in) load_x<BF16>(x, token(16 * m + i16) + (int64_t)(b0 + g) * kBlock);
        u32x4 f[NT][4];
        terms_of<BF16, HAD, NT>(x, a.sign_mask, f);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = NT - 1; s >= 0; --s)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f[s][j]),
                                                          w[r][j], p, 0, 0, 0);
          acc[m][r] += p;
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t = m0 + 16 * m + 4 * g + i, n = n0 + 16 * r + i16;
        if (t >= a.T || n >= a.N) continue;
        if (splits > 1) part[(blockIdx.z * a.T + t) * a.N + n] = acc[m][r][i];
        else store_y(a, t * a.ldy + n, acc[m][r][i]);
      }
}

// y = 2^alpha times the sum of the parts, in their order
__global__ __launch_bounds__(256) void gemv_join_kernel(const GemvArgs a,
                                                        const float* __restrict__ part,
                                                        int splits) {
  const int64_t count = a.T * a.N;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < count;
       e += (int64_t)gridDim.x * 256) {
    float v = part[e];
    int s = 1;
    for (; s + 4 <= splits; s += 4) {  // four loads on the way
      float p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = part[(s + k) * count + e];
#pragma unroll
      for (int k = 0; k < 4; ++k) v += p[k];
    }
    for (; s < splits; ++s) v += part[s * count + e];
    store_y(a, a.ldy == a.N ? e : e / a.N * a.ldy + e % a.N, v);
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

template <bool BF16, bool HAD, int NT, int RT>
hipError_t launch_direct(const GemvArgs& a) {
  const int64_t gx = (a.N + 16 * RT - 1) / (16 * RT), gy = (a.T + 15) / 16;
  hipLaunchKernelGGL((gemv_direct_kernel<BF16, HAD, NT, RT>), dim3((unsigned)gx, (unsigned)gy),
                     dim3(512), 0, (hipStream_t)a.stream, a);
  return hipGetLastError();
}

// blocks of K that a workgroup's LDS holds within `bytes`: NT terms of T tokens and the scale rows
int segment_blocks(const GemvArgs& a, int nt, int rows, int bytes) {
  const int srows = a.gw == 1 ? rows : (rows + a.gw - 1) / a.gw;
  const int64_t nb = a.K / 32, nb4 = (nb + 3) / 4 * 4;
  int64_t seg = (bytes - 20 * srows) / (64 * nt * a.T + srows) / 16 * 16;
  return (int)(seg < nb4 ? seg : nb4);
}

constexpr int kLds = 128 * 1024;         // of a workgroup, at most
constexpr int kLdsOfUnit = 160 * 1024;  // of a compute unit

// LDS of a workgroup of gemv_kernel whose segments have `seg` blocks: terms and scale bytes, later the
// waves' sums
int lds_bytes(const GemvArgs& a, int nt, int rt, int wv, int seg) {
  const int srows = a.gw == 1 ? 16 * rt : (16 * rt + a.gw - 1) / a.gw;
  const int use = nt * seg * 64 * (int)a.T + srows * scale_pitch(seg), join = wv * rt * 1024;
  return use > join ? use : join;
}

template <bool BF16, bool HAD, int NT, int RT, int WV, bool ONE = true>
hipError_t launch_gemv(const GemvArgs& a) {
  const int64_t gx = (a.N + 16 * RT - 1) / (16 * RT);
  const int seg = segment_blocks(a, NT, 16 * RT, kLds);
  hipLaunchKernelGGL((gemv_kernel<BF16, HAD, NT, RT, WV, ONE>), dim3((unsigned)gx), dim3(64 * WV),
                     lds_bytes(a, NT, RT, WV, seg), (hipStream_t)a.stream, a, seg);
  return hipGetLastError();
}

// One token: how many codes are on the way is a matter of how many waves a compute unit holds, and
// that of how many workgroups of 16 rows there are for it and how many its LDS has room for. Where it
// would hold two workgroups at most, they have 8 waves, else 4. Where a single one fills LDS and
// there are more of them than compute units, two row tiles halve the number of times that the
// activations are brought in, rotated and split. (us with 4 waves | 8 waves | 8 waves and two tiles:
// bf16 N 4096, K 8192 9.2 | 8.5 | 9.1; N 11008, K 4096 8.1 | 10.0 | 11.1; N 20480, K 28672 74 | 58 |
// 70; rotated N 16384, K 8192 20.4 | 24.7 | 22.7; fp32 N 8192, K 14336 27.8 | 21.3 | 17.9.) Of 546
// sizes (N 256 to 40960, K 512 to 28672, every type) it is 0.4% (bf16), 3.4% (rotated) and 1.1%
// (fp32) from the best of these and two tiles with 4 waves, 1.44 times at worst (rotated, K 512).
template <bool BF16, bool HAD, int NT>
hipError_t launch_one(const GemvArgs& a) {
  const int64_t wanted = (a.N + 16 * 256 - 1) / (16 * 256);
  const int room = kLdsOfUnit / lds_bytes(a, NT, 1, 4, segment_blocks(a, NT, 16, kLds));
  if (room == 1 && wanted > 1) return launch_gemv<BF16, HAD, NT, 2, 8>(a);
  if (room <= 2 || wanted <= 2) return launch_gemv<BF16, HAD, NT, 1, 8>(a);
  return launch_gemv<BF16, HAD, NT, 1, 4>(a);
}

template <bool BF16, bool HAD, int NT, int MT, int RT>
hipError_t launch_shared(const GemvArgs& a, float* part, int splits) {
  constexpr int kRows = 128 * RT;
  const int64_t gx = (a.N + kRows - 1) / kRows, gy = (a.T + 16 * MT - 1) / (16 * MT);
  hipLaunchKernelGGL((gemv_shared_kernel<BF16, HAD, NT, MT, RT>),
                     dim3((unsigned)gx, (unsigned)gy, (unsigned)splits), dim3(512), 0,
                     (hipStream_t)a.stream, a, part, splits);
  if (hipError_t e = hipGetLastError(); e != hipSuccess || splits == 1) return e;
  const int64_t blocks = (a.T * a.N + 255) / 256;
  hipLaunchKernelGGL(gemv_join_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256),
                     0, (hipStream_t)a.stream, a, part, splits);
  return hipGetLastError();
}

// All activations through LDS in one piece: for one token always (N 14336, K 4096: rotated 10.4 us,
// 14.2 read directly; fp32 11.8 and 14.8; bf16, N 8192, K 28672: 26.3 and 30.1), and for very few
// tokens that have to be rotated or split, few rows and a K that is not short, as long as two
// workgroups a compute unit hold them (4 rotated tokens, N 4096, K 4128: 8.8 us, 10.7 with
// gemv_shared_kernel; N 5120, K 512: 7.7 and 4.6; N 28672, K 1024: 15.5 and 7.5).
bool takes_lds(int64_t T, int64_t N, int64_t K, int nt) {
  return T == 1 || (nt > 1 && T * nt <= 8 && K >= 2048 && T * K * 2 * nt <= kLds / 2 &&
                    N <= 16 * 256);
}

// How a product of several tokens is taken: by gemv_shared_kernel with `tiles` tiles of 16 tokens,
// 128 `rt` rows a workgroup and K in `parts` parts (several want a workspace), or, with parts = 0, by
// gemv_direct_kernel with `rt` tiles of 16 rows.
struct Plan {
  int tiles, rt, parts;
};

// The shapes differ in how many workgroups there are, how often activations are fetched and split and
// codes converted, and in the join; which one is best changes with every size (16 bf16 tokens, K
// 4096: N 4096 7.2 us directly, 9.0 shared; K 1024, N 28672: 9.5 and 6.7; K 8192: 48.4 and 32.7; N
// 1003, K 16384: 24.2 and 12.2; 64 fp32 tokens, N 8192, K 2048: 23.1 and 12.6). So the time is
// estimated, in us, from what a workgroup does one after the other (chunks of 512 of K, in rounds of
// 256 workgroups), what the machine does in all (codes), the blocks after the last chunk, and the
// join. The constants are fitted to 2550 sizes (2 to 100 tokens, N 64 to 40960, K 256 to 28672, all
// types; every shape of either kernel timed), of which the choice is 1 to 4% from the best one on
// average, where thresholds on N and K were at 11 to 13% and up to 6 times. Of 660 other sizes from
// the same ranges it is 2.1% (bf16), 1.7% (rotated) and 0.2% (fp32) from the best; among those with
// more than 40 MB of weights 4 to 7%, 1.3 to 1.5 times at worst, where K in parts would help more
// than 128 groups too (8 bf16 tokens, N 34227, K 11456: 80.6 us, 60.3 in 8 parts of 128 rows).
// Workgroups of 7 or 16 waves for gemv_shared_kernel were no better (16 rotated tokens, N 28672, K
// 8192: 43.6 and 40.4 us, 37.4 with 8), nor more parts than one workgroup a compute unit (42.7).
double shared_time(int64_t T, int64_t N, int64_t K, int nt, int tiles, int rt, int64_t parts) {
  const int64_t groups = (N + 128 * rt - 1) / (128 * rt) * ((T + 16 * tiles - 1) / (16 * tiles));
  const int64_t wgs = groups * parts, len = (K / 512 + parts - 1) / parts, rounds = (wgs + 255) / 256;
  const int64_t rest = (K % 512 + 127) / 128;  // steps
  const double chunk = rt * (0.68 + 0.22 * tiles * nt) + tiles * (nt > 1 ? 0.28 + 0.17 * nt : 0.28);
  const double after = rest ? 1.2 + rest * rt * (0.07 + 0.3 * tiles * nt) : 0.0;
  const double join = parts > 1 ? 3.2 + 0.2e-6 * (double)(parts * T * N) : 0.0;
  return 3.2 + rounds * (len * chunk + after) + 0.33 / 256 * rt * (double)(wgs * len) + join;
}

double direct_time(int64_t T, int64_t N, int64_t K, int nt, int rt) {
  struct Cost {
    double start, turn, turn_rt, x, all, all_rt, rest, rest_rt;
  };
  constexpr Cost kCost[3] = {{2.0, 0.12, 0.51, 3.15, 0.43, 1.22, 0.45, 0.26},
                             {1.7, 2.72, 0.67, 2.87, 1.49, 0.61, 1.20, 0.44},
                             {1.6, 1.63, 1.07, 5.26, 1.27, 0.80, 1.21, 0.39}};
  const Cost& c = kCost[nt - 1];
  const int64_t wgs = (N + 16 * rt - 1) / (16 * rt) * ((T + 15) / 16), rounds = (wgs + 255) / 256;
  const int64_t chunks = K / 512, turns = (chunks + 7) / 8;  // of 8 waves
  const double x = (double)chunks / 8 * c.x * (T < 16 ? (double)T / 16 : 1.0);
  const double rest = K % 512 ? c.rest + c.rest_rt * rt : 0.0;
  return c.start + rounds * (turns * (c.turn + c.turn_rt * rt) + x + rest) +
         (double)(wgs * chunks) / 2048 * (c.all + c.all_rt * rt);
}

Plan plan_gemv(int64_t T, int64_t N, int64_t K, int nt, bool workspace) {
  Plan best{1, 1, 0};
  double least = direct_time(T, N, K, nt, 1);
  auto offer = [&](double time, const Plan& p) {
    if (time < least) {
      least = time;
      best = p;
    }
  };
  for (int rt = 2; rt <= (nt == 1 ? 4 : 2); rt *= 2)
    offer(direct_time(T, N, K, nt, rt), Plan{1, rt, 0});
  const int64_t chunks = K / 512;
  if (chunks < 1) return best;
  // More than 8 parts have two chunks at least: 16 fp32 tokens, N 1003, K 16384: 13.9 us in 16, 16.0
  // in 32; 37, K 4128: 10.8 in 8, 11.7 in 4.
  const int64_t cut = chunks <= 8 ? chunks : chunks / 2 < 8 ? 8 : chunks / 2;
  const int most_tiles = nt == 1 ? 4 : nt == 2 ? 2 : 1;  // two chunks of a tile: 32 KB of LDS a term
  for (int tiles = 1; tiles <= most_tiles && (tiles == 1 || T > 8 * tiles); tiles *= 2)
    for (int rt = 1; rt <= 2; ++rt) {
      const int64_t groups = (N + 128 * rt - 1) / (128 * rt) * ((T + 16 * tiles - 1) / (16 * tiles));
      const int64_t most = !workspace || groups > 128 ? 1 : 256 / groups < cut ? 256 / groups : cut;
      for (int64_t s = 1; s < most; s *= 2)
        offer(shared_time(T, N, K, nt, tiles, rt, s), Plan{tiles, rt, (int)s});
      offer(shared_time(T, N, K, nt, tiles, rt, most), Plan{tiles, rt, (int)most});
    }
  return best;
}

template <bool BF16, bool HAD, int NT>
hipError_t pick_gemv(const GemvArgs& a) {
  if (a.T == 1) return launch_one<BF16, HAD, NT>(a);
  if constexpr (NT > 1)
    if (takes_lds(a.T, a.N, a.K, NT)) return launch_gemv<BF16, HAD, NT, 1, 8, false>(a);
  const Plan p = plan_gemv(a.T, a.N, a.K, NT, a.part != nullptr);
  if (p.parts == 0) {
    if constexpr (NT == 1)
      if (p.rt == 4) return launch_direct<BF16, HAD, NT, 4>(a);
    return p.rt == 2 ? launch_direct<BF16, HAD, NT, 2>(a) : launch_direct<BF16, HAD, NT, 1>(a);
  }
  if constexpr (NT == 1)
    if (p.tiles == 4)
      return p.rt == 2 ? launch_shared<BF16, HAD, NT, 4, 2>(a, a.part, p.parts)
                       : launch_shared<BF16, HAD, NT, 4, 1>(a, a.part, p.parts);
  if constexpr (NT <= 2)
    if (p.tiles == 2)
      return p.rt == 2 ? launch_shared<BF16, HAD, NT, 2, 2>(a, a.part, p.parts)
                       : launch_shared<BF16, HAD, NT, 2, 1>(a, a.part, p.parts);
  return p.rt == 2 ? launch_shared<BF16, HAD, NT, 1, 2>(a, a.part, p.parts)
                   : launch_shared<BF16, HAD, NT, 1, 1>(a, a.part, p.parts);
}

// bf16 terms of an activation: fp32 values take 3; rotated bf16 ones 2 when y is bf16
int terms(bool bf16, bool hadamard, bool out_bf16) {
  return bf16 && !hadamard ? 1 : bf16 && out_bf16 ? 2 : 3;
}

}  // namespace

int64_t mx_gemv_workspace_bytes(int64_t T, int64_t N, int64_t K, bool bf16, bool hadamard,
                                bool out_bf16) {
  const int nt = terms(bf16, hadamard, out_bf16);
  if (takes_lds(T, N, K, nt)) return 0;
  const int64_t parts = plan_gemv(T, N, K, nt, true).parts;
  return parts > 1 ? parts * T * N * (int64_t)sizeof(float) : 0;
}

hipError_t mx_launch_gemv(const GemvArgs& a) {
  if (a.K == 0) {
    const int64_t blocks = (a.T * a.N + 255) / 256;
    hipLaunchKernelGGL(gemv_zero_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256),
                       0, (hipStream_t)a.stream, a);
    return hipGetLastError();
  }
  if (a.bf16 && !a.hadamard) return pick_gemv<true, false, 1>(a);
  if (a.bf16 && a.out_bf16) return pick_gemv<true, true, 2>(a);
  if (a.bf16) return pick_gemv<true, true, 3>(a);
  return a.hadamard ? pick_gemv<false, true, 3>(a) : pick_gemv<false, false, 3>(a);
}
