// lora.hip — low-rank adapters of many requests beside a shared projection, for gfx950:
//   out[t] = base[t] + s[e] B[e] (A[e] x[t]),   e = index[t], A [E][r][K], B [E][N][r].
//
// Two kernels: the first forms h = A x (fp32, in parts over K, in the workspace), the second sums the
// parts and forms base + s B h with one rounding. Tokens come in any order, so each kernel takes 64 of
// them at a time, a wave's lanes with an index each, and finds the adapters that occur among them by
// ballots: group k of a chunk is the k-th of them, whose tokens are the products' rows or columns,
// 16 at a time. An adapter's weights are read once for 64 tokens (16 in the first kernel), and a token
// meets no other adapter's weights. The grid has a group for every adapter that there may be; those
// that there are not come last in the order of launch, where they leave the others evenly spread (a
// workgroup for every adapter and chunk, in that order, took 51 us for 8192 tokens, K 4096, 8 adapters
// of rank 16: the ones with work met on few compute units).
#include "mx_device.h"
#include "mx_launch.h"

#include <type_traits>

using namespace mxd;

namespace {

constexpr int kChunk = 64;      // tokens a workgroup looks at
constexpr int kMostParts = 16;  // of K
constexpr int kSmallWaves = 16;

// tokens of a chunk with one adapter
struct Members {
  int count, adapter;  // adapter -1: tokens without one
  int first;           // of the members the workgroup has, the first one's number
  int token;           // this lane's: member number `lane`
};

// Group k of a chunk: the k-th SIZE tokens of the adapters that occur, with NONE the tokens without one
// among them (SIZE 64: an adapter's tokens are one group).
template <bool NONE, int SIZE>
__device__ __forceinline__ Members members_of(const LoraArgs& a, int chunk, int k) {
  const int lane = threadIdx.x & 63, t = chunk * kChunk + lane;
  int e = a.E;  // none
  if (t < a.T && a.E > 0) e = a.index[t];
  if (e < 0 || e > a.E) e = a.E;
  const bool counts = t < a.T && (NONE || e < a.E);
  // the lanes with this lane's adapter, from one ballot for each bit of it
  uint64_t same = __ballot(counts);
  for (int bits = 32 - __builtin_clz(a.E | 1), i = 0; i < bits; ++i) {
    const bool bit = (e >> i) & 1;
    const uint64_t ones = __ballot(bit);
    same &= bit ? ones : ~ones;
  }
  const uint64_t below = (1ull << lane) - 1;
  // the first lane of an adapter has its groups; those before it are the earlier ones' groups
  const bool leads = counts && (same & below) == 0;
  const int size = __popcll(same), groups = (size + SIZE - 1) / SIZE;
  int before = __popcll(__ballot(leads) & below);
#pragma unroll
  for (int n = 2; n <= kChunk / SIZE; ++n)
    before += __popcll(__ballot(leads && groups >= n) & below);
  const uint64_t mine = __ballot(leads && before <= k && k < before + groups);
  Members m;
  m.count = 0;
  if (mine == 0) return m;
  const int from = __builtin_ctzll(mine);
  m.adapter = __builtin_amdgcn_readlane(e, from);
  if (m.adapter == a.E) m.adapter = -1;
  m.first = SIZE * (k - __builtin_amdgcn_readlane(before, from));
  const uint64_t mask = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)same, from) |
                        (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(same >> 32), from) << 32;
  m.count = __popcll(mask);
  // members first, in their order: lane l's place among them, or behind them among the others
  const int place = (mask >> lane) & 1 ? __popcll(mask & below)
                                       : __popcll(mask) + __popcll(~mask & below);
  m.token = chunk * kChunk + __builtin_amdgcn_ds_permute(4 * place, lane);
  return m;
}

// 64 reduction indexes of 16 rows, in a wave. As operands of a product (a lane has 16 g .. 16 g + 15 of
// row i) lanes that follow one another have different rows: read that way each of a load's 16 bytes is
// a look into the cache of its own. Rows are read whole instead, 8 or 16 lanes each, and put in order
// through LDS, in an area of the wave's own.
template <bool BF16>
struct Piece {
  u32x4 w[BF16 ? 2 : 4];
};

template <bool BF16>
struct Exchange {
  static constexpr int E = BF16 ? 2 : 4, WORDS = BF16 ? 2 : 4, PER = 4 * E, ROWS = 64 / PER;
  static constexpr int PITCH = 64 * E + 16;
  typedef uint8_t Area[16 * PITCH];
  // the row of word w that this lane reads, and its byte in the 64 indexes
  static __device__ __forceinline__ int row(int w) { return ROWS * w + (threadIdx.x & 63) / PER; }
  static __device__ __forceinline__ int byte() { return 16 * (threadIdx.x & (PER - 1)); }

  static __device__ __forceinline__ Piece<BF16> operand(const Piece<BF16>& rows, uint8_t* area) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int w = 0; w < WORDS; ++w) *reinterpret_cast<u32x4*>(area + row(w) * PITCH + byte()) = rows.w[w];
    order();
    Piece<BF16> o;
#pragma unroll
    for (int w = 0; w < WORDS; ++w)
      o.w[w] = *reinterpret_cast<const u32x4*>(area + (lane & 15) * PITCH + (lane >> 4) * 16 * E + 16 * w);
    order();
    return o;
  }
  // a wave's LDS accesses complete in order; the compiler keeps them so
  static __device__ __forceinline__ void order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
};

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

// A x of 16 members (m.first ..), steps from + wave, from + wave + waves, .. of 64 up to `to`. RT: 16-row
// tiles of A; area: the wave's own.
template <bool BF16, int RT>
__device__ __forceinline__ void accumulate(const LoraArgs& a, const Members& m, int first, int from, int to,
                                           int wave, int waves, uint8_t* area, f32x4 (&acc)[RT]) {
  typedef Exchange<BF16> X;
  constexpr int E = X::E, WORDS = X::WORDS;
  const uint8_t* rows[RT][WORDS];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int w = 0; w < WORDS; ++w)
      rows[r][w] = static_cast<const uint8_t*>(a.a) + X::byte() +
                   ((int64_t)m.adapter * a.r + min(16 * r + X::row(w), a.r - 1)) * a.K * E;
  const uint8_t* x[WORDS];
#pragma unroll
  for (int w = 0; w < WORDS; ++w)
    x[w] = static_cast<const uint8_t*>(a.x) + X::byte() +
           (int64_t)__shfl(m.token, min(first + X::row(w), m.count - 1)) * a.ldx * E;
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = f32x4{0, 0, 0, 0};
  auto take = [&](const Piece<BF16>& v, const Piece<BF16>(&w)[RT]) {
    const Piece<BF16> right = X::operand(v, area);
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = multiply<BF16>(X::operand(w[r], area), right, acc[r]);
  };
  // whole steps, the next one's weights and values on their way
  const int whole = min(to, a.K / 64);
  int s = from + wave;
  Piece<BF16> v, w[RT];
  if (s < whole) {
    auto load = [&](int step, Piece<BF16>& v, Piece<BF16>(&w)[RT]) {
      const int64_t k = 64 * E * (int64_t)step;
#pragma unroll
      for (int n = 0; n < WORDS; ++n) v.w[n] = *reinterpret_cast<const u32x4*>(x[n] + k);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < WORDS; ++n) w[r].w[n] = *reinterpret_cast<const u32x4*>(rows[r][n] + k);
    };
    load(s, v, w);
    for (; s < whole; s += waves) {
      Piece<BF16> v2, w2[RT];
      load(s + waves < whole ? s + waves : s, v2, w2);
      take(v, w);
      v = v2;
#pragma unroll
      for (int r = 0; r < RT; ++r) w[r] = w2[r];
    }
  }
  if (s < to) {  // the last, K % 64 of it: zeros from there on
    const bool in = X::byte() < (a.K - 64 * s) * E;
    const int64_t k = in ? 64 * E * (int64_t)s : -X::byte();
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int n = 0; n < WORDS; ++n) {
      const u32x4 t = *reinterpret_cast<const u32x4*>(x[n] + k);
      v.w[n] = in ? t : zero;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const u32x4 y = *reinterpret_cast<const u32x4*>(rows[r][n] + k);
        w[r].w[n] = in ? y : zero;
      }
    }
    take(v, w);
  }
}

// h = A x. Grid: parts of K, chunks of tokens, groups of 16 of their tokens. The four waves take every
// fourth 64 of the part's K; their sums are joined in LDS in the waves' order.
// 2048 tokens, K 4096, rank 64: 13.1 us by the tracer, 11.2 on one set of inputs again and again. (Two or
// four 16s of tokens a workgroup, which read A once for them, and workgroups of 8 or 16 waves were tried
// while rows were read in the operands' order, not since they are read whole: 16.8 us to 17.5 and 15.0, and
// 15.7 to 18.4 and 19.8 for 256 tokens of 64 adapters, K 8192, rank 32.)
template <bool BF16, int RT>
__global__ __launch_bounds__(256) void lora_down_kernel(const LoraArgs a) {
  __shared__ __attribute__((aligned(16))) float sums[4][RT][16][20];
  __shared__ __attribute__((aligned(16))) typename Exchange<BF16>::Area area[4];
  const Members m = members_of<false, 16>(a, blockIdx.y, blockIdx.z);
  if (m.count == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4, wave = tid >> 6;
  const int steps = (a.K + 63) / 64;
  const int from = steps * blockIdx.x / gridDim.x, to = steps * (blockIdx.x + 1) / gridDim.x;
  f32x4 acc[RT];
  accumulate<BF16, RT>(a, m, m.first, from, to, wave, 4, area[wave], acc);
#pragma unroll
  for (int r = 0; r < RT; ++r) *reinterpret_cast<f32x4*>(&sums[wave][r][i][4 * g]) = acc[r];
  __syncthreads();
  for (int e = tid; e < RT * 256; e += 256) {
    const int col = e / (16 * RT), row = e % (16 * RT);  // a token's r values in a row
    const int token = __shfl(m.token, min(m.first + col, 63));
    if (m.first + col < m.count && row < a.r) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) v += sums[w][row / 16][col][row % 16];
      a.h[((int64_t)blockIdx.x * a.T + token) * a.r + row] = v;
    }
  }
}

// Four values of a row from `at` on, `n` of them inside it, as they are in memory (bf16: two words);
// WIDE: all four, at an address for one load
template <bool BF16, bool WIDE>
__device__ __forceinline__ u32x4 load4(const void* p, int64_t at, int n) {
  if constexpr (WIDE) {
    if constexpr (!BF16) return *reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + at);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
    return u32x4{w.x, w.y, 0, 0};
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) {
        if constexpr (BF16) w[i / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[at + i] << (16 * (i % 2));
        else w[i] = static_cast<const uint32_t*>(p)[at + i];
      }
    return u32x4{w[0], w[1], w[2], w[3]};
  }
}

template <bool BF16>
__device__ __forceinline__ f32x4 values4(const u32x4& w) {
  if constexpr (!BF16) return __builtin_bit_cast(f32x4, w);
  return f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u),
               __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xFFFF0000u)};
}

template <bool BF16, bool WIDE>
__device__ __forceinline__ void store4(void* p, int64_t at, int n, const f32x4& v) {
  const bf16x2_t lo = {(__bf16)v[0], (__bf16)v[1]}, hi = {(__bf16)v[2], (__bf16)v[3]};
  const uint32_t w[2] = {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
  if constexpr (WIDE) {
    if constexpr (BF16) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<f32x4*>(static_cast<float*>(p) + at) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) {
        if constexpr (BF16) static_cast<uint16_t*>(p)[at + i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
        else static_cast<float*>(p)[at + i] = v[i];
      }
  }
}

// out = base + s B h. Grid: slabs of B's rows, chunks of tokens, adapters of a chunk and its tokens
// without one. A wave has 64 rows at a time: tile q's column i is row 4 i + q of them, so that a lane has
// four neighbours of an output row and 16 lanes 64 of them, and the tokens are the products' rows. h goes
// in as three bf16 terms that add up to the fp32 value (fp32 weights: as it is). base and B are on their
// way while h is summed. 2048 tokens, N 14336, rank 64: 43 us, 4.1 TB/s (56 from cold memory).
template <bool BF16, int RT>
struct Up {
  static constexpr int JS = BF16 ? 32 : 16;                         // of the rank in a product
  static constexpr int W = BF16 && RT == 1 ? 32 : 16 * RT;          // the rank, filled up with zeros
  static constexpr int JT = W / JS, NT = BF16 ? 3 : 1;
  typedef typename std::conditional<BF16, uint16_t, float>::type term_t;
  struct Shared {
    term_t h[NT][kChunk][W + (BF16 ? 8 : 4)];
  };

  // h of the members, as the products take it: zeros from r to W; rows behind the members' are not set, a
  // product's other rows do not depend on them. Four lanes have four of a token's r values, each every
  // fourth part of K, and join them as (0 + 1) + (2 + 3); a wave has 16 such values a turn, and the loads of
  // TURNS turns and ROUNDS times 4 parts are under way at once.
  template <int ROUNDS, int TURNS>
  static __device__ __forceinline__ void sum_parts(const LoraArgs& a, const Members& m, float scale,
                                                   Shared& sh) {
    const int tid = threadIdx.x, part = tid & 3, fours = a.r / 4, all = m.count * fours;
    const int64_t stride = (int64_t)a.T * a.r;
    for (int e0 = 0; e0 < all; e0 += 64 * TURNS) {
      f32x4 v[TURNS][ROUNDS];
      int col[TURNS], j[TURNS];
#pragma unroll
      for (int k = 0; k < TURNS; ++k) {
        const int e = min(e0 + 64 * k + tid / 4, all - 1);
        col[k] = e / fours;
        j[k] = 4 * (e - col[k] * fours);
        const float* p = a.h + (int64_t)__shfl(m.token, col[k]) * a.r + j[k];
        if (k == 0 || e0 + 64 * k < all) {
#pragma unroll
          for (int s = 0; s < ROUNDS; ++s)
            v[k][s] = *reinterpret_cast<const f32x4*>(p + min(4 * s + part, a.parts - 1) * stride);
        }
      }
#pragma unroll
      for (int k = 0; k < TURNS; ++k) {
        if (k > 0 && e0 + 64 * k >= all) break;
        float one = 0.0f;  // this lane's of the four
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float own = 0.0f;
#pragma unroll
          for (int s = 0; s < ROUNDS; ++s) own += 4 * s + part < a.parts ? v[k][s][x] : 0.0f;
          const float pair = own + dpp_f32<kQuadXor1>(own);
          const float sum = pair + dpp_f32<kQuadXor2>(pair);
          if (x == part) one = sum * scale;
        }
        put(sh, col[k], j[k] + part, one);
      }
    }
    const int rest = W - a.r;
    for (int e = tid; e < m.count * rest; e += 256) put(sh, e / rest, a.r + e % rest, 0.0f);
  }

  static __device__ __forceinline__ void put(Shared& sh, int col, int j, float v) {
    if constexpr (BF16) {
      uint32_t o[3];
      split_pair<3>(v, 0.0f, o);
#pragma unroll
      for (int n = 0; n < 3; ++n) sh.h[n][col][j] = (uint16_t)o[n];
    } else {
      sh.h[0][col][j] = v;
    }
  }

  // Four neighbours of base's rows of tile `tile`'s tokens 4 g .., at n. BASE: 0 none, 1 fp32, 2 bf16; WIDE:
  // all inside the row, at an address for one load.
  template <int BASE, bool WIDE>
  static __device__ __forceinline__ void load_base(const LoraArgs& a, const Members& m, int tile, int n,
                                                   u32x4 (&base)[4]) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t token = __shfl(m.token, min(16 * tile + 4 * g + r, m.count - 1));
      base[r] = BASE == 0 ? u32x4{0, 0, 0, 0} : load4<BASE == 2, WIDE>(a.base, token * a.ldb + n, a.N - n);
    }
  }
  static __device__ __forceinline__ void first_base(const LoraArgs& a, const Members& m, bool wide, int n,
                                                    u32x4 (&base)[4]) {
    if (!a.base) load_base<0, false>(a, m, 0, n, base);
    else if (a.base_bf16) wide ? load_base<2, true>(a, m, 0, n, base) : load_base<2, false>(a, m, 0, n, base);
    else wide ? load_base<1, true>(a, m, 0, n, base) : load_base<1, false>(a, m, 0, n, base);
  }

  // B's rows n .. n + 63, four neighbouring lanes a row's 64 bytes; then each lane's rows n + 4 i .. by
  // an exchange of registers. Read in that order directly, neighbouring lanes have different rows and
  // each 16 bytes are a line lookup of their own (2048 tokens of 64 adapters, N and K 4096, rank 16: 85
  // us both kernels, 74.5 so; one token, N 14336: 8.5, 7.8; 2048 tokens of 4 adapters, rank 64: level).
  static __device__ __forceinline__ void load_weights(const LoraArgs& a, const Members& m, int n,
                                                      u32x4 (&w)[JT][4]) {
    const int lane = threadIdx.x & 63, g = lane & 3;
    n += 4 * (lane >> 2);
#pragma unroll
    for (int k = 0; k < JT; ++k) {
      const int j = k * JS + (BF16 ? 8 : 4) * g;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t row = (int64_t)m.adapter * a.N + min(n + q, a.N - 1);
        const u32x4 t = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.b) +
                                                        (row * a.r + (j < a.r ? j : 0)) * (BF16 ? 2 : 4));
        w[k][q] = j < a.r ? t : u32x4{0, 0, 0, 0};
      }
    }
  }

  static __device__ __forceinline__ void order_weights(u32x4 (&w)[JT][4]) {
    const int lane = threadIdx.x & 63, from = 4 * (4 * (lane & 15) + (lane >> 4));
#pragma unroll
    for (int k = 0; k < JT; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[k][q][e] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)w[k][q][e]);
  }

  // 64 rows of B (those at n = n0 + 4 i ..), all members; base holds the first tile's
  template <int BASE, bool OUT, bool WIDE>
  static __device__ __forceinline__ void slab(const LoraArgs& a, const Members& m, const Shared& sh, int n,
                                              const u32x4 (&w)[JT][4], u32x4 (&base)[4]) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4, tiles = (m.count + 15) / 16;
    for (int t = 0; t < tiles; ++t) {
      f32x4 v[4], acc[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[r] = values4<BASE == 2>(base[r]);
        acc[r] = f32x4{0, 0, 0, 0};
      }
      if (t + 1 < tiles) load_base<BASE, WIDE>(a, m, t + 1, n, base);
      if (m.adapter >= 0) {
#pragma unroll
        for (int k = 0; k < JT; ++k) {
          const int j = k * JS + (BF16 ? 8 : 4) * g;
          if constexpr (BF16) {
#pragma unroll
            for (int e = 2; e >= 0; --e) {
              const bf16x8_t x = *reinterpret_cast<const bf16x8_t*>(&sh.h[e][16 * t + i][j]);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    x, __builtin_bit_cast(bf16x8_t, w[k][q]), acc[q], 0, 0, 0);
            }
          } else {
            const f32x4 x = *reinterpret_cast<const f32x4*>(&sh.h[0][16 * t + i][j]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                acc[q] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], __uint_as_float(w[k][q][e]), acc[q],
                                                              0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int at = 16 * t + 4 * g + r;
        const int64_t token = __shfl(m.token, min(at, 63));
#pragma unroll
        for (int q = 0; q < 4; ++q) v[r][q] += acc[q][r];
        if (at < m.count) store4<OUT, WIDE>(a.out, token * a.ldo + n, a.N - n, v[r]);
      }
    }
  }

  template <bool WIDE>
  static __device__ __forceinline__ void any_slab(const LoraArgs& a, const Members& m, const Shared& sh,
                                                  int n, const u32x4 (&w)[JT][4], u32x4 (&v)[4]) {
    const int base = !a.base ? 0 : a.base_bf16 ? 2 : 1;
    if (a.out_bf16) {
      if (base == 1) slab<1, true, WIDE>(a, m, sh, n, w, v);
      else if (base == 2) slab<2, true, WIDE>(a, m, sh, n, w, v);
      else slab<0, true, WIDE>(a, m, sh, n, w, v);
    } else {
      if (base == 1) slab<1, false, WIDE>(a, m, sh, n, w, v);
      else if (base == 2) slab<2, false, WIDE>(a, m, sh, n, w, v);
      else slab<0, false, WIDE>(a, m, sh, n, w, v);
    }
  }
};

template <bool BF16, int RT>
__global__ __launch_bounds__(256) void lora_up_kernel(const LoraArgs a) {
  typedef Up<BF16, RT> U;
  __shared__ __attribute__((aligned(16))) typename U::Shared sh;
  const Members m = members_of<true, kChunk>(a, blockIdx.y, blockIdx.z);
  if (m.count == 0 || (m.adapter < 0 && a.in_place)) return;
  const int tid = threadIdx.x, i = tid & 15;
  int n0 = (blockIdx.x * a.slabs * 4 + (tid >> 6)) * 64;
  u32x4 w[U::JT][4];
  const bool rows_wide = a.out_wide && (!a.base || a.base_wide);
  u32x4 base[4];
  if (n0 < a.N) U::first_base(a, m, rows_wide && n0 + 64 <= a.N, n0 + 4 * i, base);
  if (m.adapter >= 0) {
    if (n0 < a.N) U::load_weights(a, m, n0, w);
    const float scale = a.scaling ? a.scaling[m.adapter] : 1.0f;
    if (a.parts <= 4) U::template sum_parts<1, (RT >= 4 ? 8 : 4)>(a, m, scale, sh);
    else U::template sum_parts<kMostParts / 4, 2>(a, m, scale, sh);
    __syncthreads();
  }
  for (int slab = 0; slab < a.slabs && n0 < a.N; ++slab, n0 += 256) {
    const int n = n0 + 4 * i;
    const bool wide = rows_wide && n0 + 64 <= a.N;
    if (slab > 0) {
      U::first_base(a, m, wide, n, base);
      if (m.adapter >= 0) U::load_weights(a, m, n0, w);
    }
    if (m.adapter >= 0) U::order_weights(w);
    if (wide) U::template any_slab<true>(a, m, sh, n, w, base);
    else U::template any_slab<false>(a, m, sh, n, w, base);
  }
}

// Both in one launch, without a workspace, for a few tokens (see small_call): a workgroup of 16 waves
// forms h of its adapter's tokens for itself and then 1024 outputs.
__global__ __launch_bounds__(64 * kSmallWaves) void lora_small_kernel(const LoraArgs a) {
  constexpr bool BF16 = true;
  constexpr int RT = 1;
  typedef Up<BF16, RT> U;
  __shared__ __attribute__((aligned(16))) typename U::Shared sh;
  // exchanged rows, then the waves' sums
  __shared__ __attribute__((aligned(16))) union {
    typename Exchange<BF16>::Area area[kSmallWaves];
    float sums[kSmallWaves][16][20];
  } part;
  const Members m = members_of<true, kChunk>(a, 0, blockIdx.y);
  if (m.count == 0 || (m.adapter < 0 && a.in_place)) return;
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4, wave = tid >> 6;
  const int n0 = (blockIdx.x * kSmallWaves + wave) * 64, n = n0 + 4 * i;
  const bool wide = a.out_wide && (!a.base || a.base_wide) && n0 + 64 <= a.N;
  u32x4 base[4], w[U::JT][4];
  if (n0 < a.N) U::first_base(a, m, wide, n, base);
  if (m.adapter >= 0) {
    if (n0 < a.N) U::load_weights(a, m, n0, w);
    const float scale = a.scaling ? a.scaling[m.adapter] : 1.0f;
    f32x4 acc[RT];
    accumulate<BF16, RT>(a, m, 0, 0, (a.K + 63) / 64, wave, kSmallWaves, part.area[wave], acc);
    __syncthreads();
    *reinterpret_cast<f32x4*>(&part.sums[wave][i][4 * g]) = acc[0];
    __syncthreads();
    for (int e = tid; e < 16 * U::W; e += 64 * kSmallWaves) {
      const int col = e / U::W, row = e % U::W;
      float v = 0.0f;
      if (row < a.r) {
#pragma unroll
        for (int k = 0; k < kSmallWaves; ++k) v += part.sums[k][col][row];
      }
      U::put(sh, col, row, v * scale);
    }
    __syncthreads();
  }
  if (n0 >= a.N) return;
  if (m.adapter >= 0) U::order_weights(w);
  if (wide) U::template any_slab<true>(a, m, sh, n, w, base);
  else U::template any_slab<false>(a, m, sh, n, w, base);
}

template <bool BF16, int RT>
hipError_t launch(const LoraArgs& a) {
  const unsigned chunks = (unsigned)((a.T + kChunk - 1) / kChunk);
  if (a.K > 0 && a.E > 0) {
    // adapters that a chunk may have, and their 16s of tokens
    const int tokens = a.T < kChunk ? a.T : kChunk, most = a.E < tokens ? a.E : tokens;
    const int groups = most + (tokens - most) / 16;
    hipLaunchKernelGGL((lora_down_kernel<BF16, RT>), dim3(a.parts, chunks, groups), dim3(256), 0,
                       (hipStream_t)a.stream, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  const int slab = 256 * a.slabs;
  hipLaunchKernelGGL((lora_up_kernel<BF16, RT>),
                     dim3((unsigned)((a.N + slab - 1) / slab), chunks, a.groups), dim3(256), 0,
                     (hipStream_t)a.stream, a);
  return hipGetLastError();
}

hipError_t launch_small(const LoraArgs& a) {
  const int slab = 64 * kSmallWaves;
  hipLaunchKernelGGL(lora_small_kernel, dim3((unsigned)((a.N + slab - 1) / slab), a.groups),
                     dim3(64 * kSmallWaves), 0, (hipStream_t)a.stream, a);
  return hipGetLastError();
}

template <bool BF16>
hipError_t pick(const LoraArgs& a) {
  if (a.r <= 16) return launch<BF16, 1>(a);
  if (a.r <= 32) return launch<BF16, 2>(a);
  if (a.r <= 64) return launch<BF16, 4>(a);
  return launch<BF16, 8>(a);
}

// Parts of K, so that the groups of up to 16 tokens with one adapter that there may be make about 512
// workgroups; a part has 4 steps of 64 at least, one for each wave.
int parts_of(int64_t T, int64_t K, int64_t E) {
  const int64_t tiles = (T + 15) / 16, apart = E < T ? E : T, groups = tiles > apart ? tiles : apart;
  const int64_t steps = (K + 63) / 64, most = steps < 8 ? 1 : steps < 4 * kMostParts ? steps / 4 : kMostParts;
  const int64_t want = groups > 0 ? (512 + groups - 1) / groups : 1;
  return (int)(want < most ? want : most);
}

// One launch: up to 16 bf16 tokens, rank 16 at most, K up to 4096, and no more workgroups than compute
// units. It has the device for as long as the two kernels (one token, N 14336, K 4096: 8.4 us, 7.8;
// 16 tokens of 16 adapters: 9.0, 9.9; K 2048, N 512: 5.8, 7.5) and spares the host a launch and a workspace
// (13.7 us a call, 9 so). Beyond, each workgroup's own h costs more than the second launch (K 8192,
// N 8192: 10.7 us, 7.9; 64 tokens of 64 adapters, N 14336, K 4096: 25, 20; rank 32: 11.0, 8.2; fp32, rank
// 16: 14.8, 8.3).
bool small_call(bool bf16, int64_t T, int64_t N, int64_t K, int64_t E, int64_t r) {
  return bf16 && T <= 16 && r <= 16 && K <= 4096 && (E < T ? E : T) * ((N + 1023) / 1024) <= 256;
}

}  // namespace

int64_t mx_lora_workspace_bytes(bool bf16, int64_t T, int64_t N, int64_t K, int64_t E, int64_t r) {
  if (small_call(bf16, T, N, K, E, r)) return 0;
  return parts_of(T, K, E) * T * r * (int64_t)sizeof(float);
}

hipError_t mx_launch_lora(LoraArgs a) {
  a.parts = a.K > 0 ? parts_of(a.T, a.K, a.E) : 0;
  a.small = a.K > 0 && a.E > 0 && small_call(a.bf16, a.T, a.N, a.K, a.E, a.r);
  const int tokens = a.T < kChunk ? a.T : kChunk;
  a.groups = a.E < tokens ? a.E + 1 : tokens;  // adapters of a chunk, and its tokens without one
  // A workgroup sums h once for 256, 512 or 1024 outputs: as many as leave 448 workgroups, if every
  // eighth adapter occurs in a chunk (both kernels, K 4096: 2048 tokens of 64 adapters, N 4096, rank 16: 110,
  // 86 and 74 us; 1024 tokens of 4, N 4096, rank 128: 40, 44 and 56; 2048 tokens of 4, N 14336, rank 64: 67,
  // 67 and 69, where the rule takes the last; 8192 of 8, N 4096, rank 16: 68, 73 and 68).
  const int64_t chunks = (a.T + kChunk - 1) / kChunk, slabs = (a.N + 255) / 256;
  const int64_t apart = a.E < 16 ? 1 : a.E < kChunk ? a.E / 8 : kChunk / 8;
  a.slabs = 1;
  while (a.slabs < 4 && chunks * slabs * apart >= 448 * 2 * a.slabs) a.slabs *= 2;
  if (a.small) return launch_small(a);
  return a.bf16 ? pick<true>(a) : pick<false>(a);
}
