// lora.hip — low-rank adapters of many requests beside a shared projection, for gfx950:
//   out[t] = base[t] + s[e] B[e] (A[e] x[t]),   e = index[t], A [E][r][K], B [E][N][r].
//
// Two kernels: the first forms h = A x (fp32, in parts over K, in the workspace), the second sums the
// parts and forms base + s B h with one rounding. Tokens come in any order, so each kernel takes 64 of
// them at a time (a wave's lanes hold their indexes) and gives every adapter that occurs among them
// workgroups of its own: a ballot finds its tokens, 16 of which make a matrix product's columns.
// An adapter's weights are read once for 64 tokens, and a token meets no other adapter's weights.
// With few tokens the candidates are the tokens (the first of an adapter counts), with few adapters
// the adapters.
#include "mx_device.h"
#include "mx_launch.h"

using namespace mxd;

namespace {

constexpr int kChunk = 64;  // tokens a workgroup looks at

// the tokens of chunk blockIdx.z that the workgroup has
struct Members {
  int count, adapter;  // adapter -1: tokens without one
  int token;           // this lane's: member number `lane` of them
};

// Candidate c is adapter c, or with by_token the adapter of the chunk's token c if no earlier one
// has it; c == candidates: the tokens without an adapter.
__device__ __forceinline__ Members members_of(const LoraArgs& a, int c) {
  const int lane = threadIdx.x & 63, t = blockIdx.z * kChunk + lane;
  int e = -2;  // no token
  if (t < a.T) {
    e = a.E > 0 ? a.index[t] : -1;
    if (e < 0 || e >= a.E) e = -1;
  }
  Members m;
  m.adapter = c == a.candidates ? -1 : a.by_token ? __shfl(e, c) : c;
  m.adapter = __builtin_amdgcn_readfirstlane(m.adapter);
  const uint64_t mask = __ballot(e == m.adapter);
  m.count = __popcll(mask);
  if (c < a.candidates && a.by_token && (m.adapter < 0 || __builtin_ctzll(mask | (1ull << 63)) != c))
    m.count = 0;
  // members first, in their order: lane l's place among them, or behind them among the others
  const uint64_t below = (1ull << lane) - 1;
  const int place = (mask >> lane) & 1 ? __popcll(mask & below)
                                       : __popcll(mask) + __popcll(~mask & below);
  m.token = blockIdx.z * kChunk + __builtin_amdgcn_ds_permute(4 * place, lane);
  return m;
}

// A lane's 16 reduction indexes of 64 (16 g .. 16 g + 15) of one row, zeros from `left` on (a
// multiple of 8)
template <bool BF16>
struct Piece {
  u32x4 w[BF16 ? 2 : 4];
};

template <bool BF16>
__device__ __forceinline__ Piece<BF16> load_piece(const uint8_t* p, int left) {
  constexpr int PER = BF16 ? 8 : 4;
  Piece<BF16> o;
#pragma unroll
  for (int i = 0; i < (BF16 ? 2 : 4); ++i)
    o.w[i] = i * PER < left ? reinterpret_cast<const u32x4*>(p)[i] : u32x4{0, 0, 0, 0};
  return o;
}

// acc += a b^T over a piece: bf16 two products of 32, fp32 sixteen of 4 (lane group g's value e of
// word w is index 16 g + 4 w + e on either side)
template <bool BF16>
__device__ __forceinline__ f32x4 multiply(const Piece<BF16>& a, const Piece<BF16>& b, f32x4 acc) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.w[i]),
                                                    __builtin_bit_cast(bf16x8_t, b.w[i]), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w[i][e]),
                                                   __uint_as_float(b.w[i][e]), acc, 0, 0, 0);
  }
  return acc;
}

// h = A x. Grid: parts of K, candidates, chunks of tokens. The four waves take every fourth 64 of the
// part's K; their sums are joined in LDS in the waves' order. RT: 16-row tiles of A.
template <bool BF16, int RT>
__global__ __launch_bounds__(256) void lora_down_kernel(const LoraArgs a) {
  __shared__ __attribute__((aligned(16))) float sums[4][RT][16][20];
  const Members m = members_of(a, blockIdx.y);
  if (m.count == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4, wave = tid >> 6;
  constexpr int E = BF16 ? 2 : 4, TT = kChunk / 16;
  const int steps = (a.K + 63) / 64;
  const int from = (int)((int64_t)steps * blockIdx.x / gridDim.x);
  const int to = (int)((int64_t)steps * (blockIdx.x + 1) / gridDim.x);
  const int tiles = (m.count + 15) / 16;
  const uint8_t* rows[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
    rows[r] = static_cast<const uint8_t*>(a.a) +
              ((int64_t)m.adapter * a.r + min(16 * r + i, a.r - 1)) * a.K * E;
  const uint8_t* tokens[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t)
    tokens[t] = static_cast<const uint8_t*>(a.x) +
                (int64_t)__shfl(m.token, min(16 * t + i, m.count - 1)) * a.ldx * E;
  f32x4 acc[TT][RT];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[t][r] = f32x4{0, 0, 0, 0};
  for (int s = from + wave; s < to; s += 4) {
    const int k = 64 * s + 16 * g, left = a.K - k;
    Piece<BF16> w[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) w[r] = load_piece<BF16>(rows[r] + (int64_t)k * E, left);
#pragma unroll
    for (int t = 0; t < TT; ++t)
      if (t < tiles) {
        const Piece<BF16> x = load_piece<BF16>(tokens[t] + (int64_t)k * E, left);
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[t][r] = multiply<BF16>(w[r], x, acc[t][r]);
      }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
    if (t < tiles) {
      __syncthreads();
#pragma unroll
      for (int r = 0; r < RT; ++r) *reinterpret_cast<f32x4*>(&sums[wave][r][i][4 * g]) = acc[t][r];
      __syncthreads();
      for (int e = tid; e < RT * 256; e += 256) {
        const int col = e / (16 * RT), row = e % (16 * RT);  // a token's r values in a row
        const int token = __shfl(m.token, min(16 * t + col, 63));
        if (16 * t + col < m.count && row < a.r) {
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < 4; ++w) v += sums[w][row / 16][col][row % 16];
          a.h[((int64_t)blockIdx.x * a.T + token) * a.r + row] = v;
        }
      }
    }
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  return static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store1(void* p, bool bf16, int64_t i, float v) {
  if (bf16) {
    const __bf16 b = (__bf16)v;
    static_cast<uint16_t*>(p)[i] = __builtin_bit_cast(uint16_t, b);
  } else {
    static_cast<float*>(p)[i] = v;
  }
}

// 16 values of a row: n from `at` on, `n` of them inside it; whole and aligned rows by 16 bytes
__device__ __forceinline__ void load16(const void* p, bool bf16, bool wide, int64_t at, int n, float (&v)[16]) {
  if (wide && n >= 16) {
    if (bf16) {
      const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at);
      float t[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        widen_bf16x8(q[i], t);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * i + j] = t[j];
      }
    } else {
      const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 t = q[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] = t[j];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i < n ? bf16 ? load1<true>(p, at + i) : load1<false>(p, at + i) : 0.0f;
  }
}

__device__ __forceinline__ void store16(void* p, bool bf16, bool wide, int64_t at, int n, const float (&v)[16]) {
  if (wide && n >= 16) {
    if (bf16) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bf16x2_t t = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
        w[i] = __builtin_bit_cast(uint32_t, t);
      }
      u32x4* q = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + at);
      q[0] = u32x4{w[0], w[1], w[2], w[3]};
      q[1] = u32x4{w[4], w[5], w[6], w[7]};
    } else {
      f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) store1(p, bf16, at + i, v[i]);
  }
}

// out = base + s B h. Grid: slabs of 256 rows of B, candidates and the tokens without an adapter,
// chunks of tokens. A wave has 64 rows: tile q's row i is row 16 (i / 4) + 4 q + i % 4 of them, so that
// a lane ends up with 16 neighbours of a token's output. h goes in as three bf16 terms that add up
// to the fp32 value (fp32 weights: as it is).
template <bool BF16, int RT>
__global__ __launch_bounds__(256) void lora_up_kernel(const LoraArgs a) {
  constexpr int TT = kChunk / 16, PAD = 16 * RT + 4, JS = BF16 ? 32 : 16;
  __shared__ __attribute__((aligned(16))) float h[kChunk][PAD];
  const Members m = members_of(a, blockIdx.y);
  if (m.count == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 256 + (tid >> 6) * 64;
  const int tiles = (m.count + 15) / 16;
  f32x4 acc[TT][4];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[t][q] = f32x4{0, 0, 0, 0};
  if (m.adapter >= 0) {
    const float scale = a.scaling ? a.scaling[m.adapter] : 1.0f;
    for (int e0 = 0; e0 < 16 * tiles * 16 * RT; e0 += 256) {
      const int e = e0 + tid, col = e / (16 * RT), j = e % (16 * RT);
      const int token = __shfl(m.token, min(col, m.count - 1));
      float v = 0.0f;
      if (col < m.count && j < a.r)
        for (int s = 0; s < a.parts; ++s) v += a.h[((int64_t)s * a.T + token) * a.r + j];
      if (col < kChunk) h[col][j] = v * scale;
    }
    __syncthreads();
    if (n0 >= a.N) return;
    const uint8_t* rows[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      rows[q] = static_cast<const uint8_t*>(a.b) +
                ((int64_t)m.adapter * a.N + min(n0 + 16 * (i >> 2) + 4 * q + (i & 3), a.N - 1)) * a.r *
                    (BF16 ? 2 : 4);
    for (int j0 = 0; j0 < a.r; j0 += JS) {
      const int j = j0 + (BF16 ? 8 : 4) * g;
      u32x4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = j < a.r ? *reinterpret_cast<const u32x4*>(rows[q] + j * (BF16 ? 2 : 4)) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < tiles) {
          if constexpr (BF16) {
            float v[8];
            // columns past r were never written beyond the tile's width
            if (j < 16 * RT) {
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = h[16 * t + i][j + e];
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            }
            uint32_t o[4][3];
#pragma unroll
            for (int e = 0; e < 4; ++e) split_pair<3>(v[2 * e], v[2 * e + 1], o[e]);
#pragma unroll
            for (int n = 2; n >= 0; --n) {
              const bf16x8_t x = __builtin_bit_cast(bf16x8_t, u32x4{o[0][n], o[1][n], o[2][n], o[3][n]});
#pragma unroll
              for (int q = 0; q < 4; ++q)
                acc[t][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w[q]), x,
                                                                    acc[t][q], 0, 0, 0);
            }
          } else {
            const f32x4 v = *reinterpret_cast<const f32x4*>(&h[16 * t + i][j]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                acc[t][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[q][e]), v[e], acc[t][q],
                                                                 0, 0, 0);
          }
        }
    }
  } else if (n0 >= a.N || a.in_place) {
    return;
  }
  const int n = n0 + 16 * g, left = a.N - n;
#pragma unroll
  for (int t = 0; t < TT; ++t)
    if (t < tiles) {
      const int64_t token = __shfl(m.token, min(16 * t + i, m.count - 1));
      if (16 * t + i < m.count && left > 0) {
        float v[16];
        if (a.base)
          load16(a.base, a.base_bf16, a.base_wide, token * a.ldb + n, left, v);
        else
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * q + e] += acc[t][q][e];
        store16(a.out, a.out_bf16, a.out_wide, token * a.ldo + n, left, v);
      }
    }
}

template <bool BF16, int RT>
hipError_t launch(const LoraArgs& a) {
  const unsigned chunks = (unsigned)((a.T + kChunk - 1) / kChunk);
  if (a.K > 0 && a.E > 0) {
    hipLaunchKernelGGL((lora_down_kernel<BF16, RT>), dim3(a.parts, a.candidates, chunks), dim3(256), 0,
                       (hipStream_t)a.stream, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((lora_up_kernel<BF16, RT>),
                     dim3((unsigned)((a.N + 255) / 256), a.candidates + 1, chunks), dim3(256), 0,
                     (hipStream_t)a.stream, a);
  return hipGetLastError();
}

template <bool BF16>
hipError_t pick(const LoraArgs& a) {
  if (a.r <= 16) return launch<BF16, 1>(a);
  if (a.r <= 32) return launch<BF16, 2>(a);
  if (a.r <= 64) return launch<BF16, 4>(a);
  return launch<BF16, 8>(a);
}

// workgroups that look for members: the adapters, or the tokens of a chunk if they are fewer
int candidates(int64_t T, int64_t E) {
  const int64_t tokens = T < kChunk ? T : kChunk;
  return (int)(E <= tokens ? E : tokens);
}

int parts_of(int64_t T, int64_t K, int64_t E) {
  const int64_t groups = candidates(T, E) * ((T + kChunk - 1) / kChunk);
  const int64_t steps = (K + 63) / 64, most = steps / 4 > 0 ? steps / 4 : 1;
  const int64_t want = groups > 0 ? (512 + groups - 1) / groups : 1;
  return (int)(want < most ? want : most);
}

}  // namespace

int64_t mx_lora_workspace_bytes(int64_t T, int64_t K, int64_t E, int64_t r) {
  return parts_of(T, K, E) * T * r * (int64_t)sizeof(float);
}

hipError_t mx_launch_lora(LoraArgs a) {
  a.candidates = candidates(a.T, a.E);
  a.by_token = a.candidates < a.E;
  a.parts = a.K > 0 ? parts_of(a.T, a.K, a.E) : 0;
  return a.bf16 ? pick<true>(a) : pick<false>(a);
}
