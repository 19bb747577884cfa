// cache.hip — keys and values in a paged cache of 8-bit codes for gfx950: written as they come, read
// back, and attended to.
//
// The cache is blocks of 32 tokens x one head: block (page * heads + head) * (page_size / 32) + i
// holds 32 * dim code bytes (E4M3 or E5M2) of keys and as many of values, and one E8M0 scale byte
// each. Key codes lie token after token ([32][dim]: the scores sum over dim), value codes channel
// after channel ([dim][32]: the output sums over tokens), so that either product finds its
// reduction index contiguous in memory and the attention transposes nothing.
//
// A block's scale serves all its 32 tokens, and tokens come one at a time: a block that already
// holds some takes the larger of its scale and the new tokens' one. Scales are powers of two and
// codes floating, so older codes are rounded again only where they fall below the least normal.
#include "mx_device.h"
#include "mx_launch.h"

#include <type_traits>

using namespace mxd;

namespace {

// the sequence of a call's rows: `n` newest tokens at rows row0 .. , `length` tokens in all
struct Sequence {
  int row0, n, length;
};

// Tables are device data: whatever they hold, rows stay inside [0, T) and pages inside the cache.
__device__ __forceinline__ Sequence sequence_from(int from, int to, int length, int rows) {
  Sequence s;
  s.row0 = min(max(from, 0), rows);
  s.n = max(min(to, rows) - s.row0, 0);
  s.length = min(max(length, 0), 0x7FFF0000);  // positions of its last block stay in 32 bits
  return s;
}
__device__ __forceinline__ Sequence sequence_of(const CacheArgs& c, int b, int rows) {
  return c.offsets ? sequence_from(c.offsets[b], c.offsets[b + 1], c.lengths[b], rows)
                   : sequence_from(b, b + 1, c.lengths[b], rows);
}

// the place in a page table of the page that holds positions 32 bn ..: bn / page_blocks by a product,
// exact for bn < 2^26 and page_blocks <= 64
__device__ __forceinline__ int slot_of(const CacheArgs& c, int bn) {
  return c.page_blocks == 1 ? bn : (int)__umulhi((uint32_t)bn, c.page_magic);
}

// The block that holds positions 32 bn .. of sequence b, -1 where the table has no such page.
__device__ __forceinline__ int64_t block_of(const CacheArgs& c, const int32_t* pages, int b, int bn,
                                            int head) {
  const int slot = slot_of(c, bn);
  if (bn < 0 || slot >= c.table_width) return -1;
  const int page = pages[(int64_t)b * c.table_width + slot];
  if (page < 0 || page >= c.n_pages) return -1;
  return ((int64_t)page * c.heads + head) * c.page_blocks + (bn - slot * c.page_blocks);
}

// Which block of which sequence a workgroup of mx_cache_write or mx_cache_read has. A sequence whose
// rows begin at o takes the units from o / 32 + 2 b on: n tokens touch (n + 30) / 32 + 1 blocks at
// most, which fits below the next sequence's first unit.
struct Piece {
  int b, bn, lo, hi;  // slots lo .. hi - 1 of the block are rows row .. of the call
  int row;
};

__device__ __forceinline__ bool piece_of(const CacheArgs& c, int unit, int rows, Piece& o) {
  __shared__ int found[4];
  int b = unit, j = 0;
  Sequence s;
  if (c.offsets) {
    if (threadIdx.x == 0) found[0] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < c.seqs; i += blockDim.x) {
      const int from = c.offsets[i], to = c.offsets[i + 1], length = c.lengths[i];
      if ((from >> 5) + 2 * i <= unit && unit < (to >> 5) + 2 * i + 2) {
        found[0] = i;
        found[1] = from;
        found[2] = to;
        found[3] = length;
      }
    }
    __syncthreads();
    b = __builtin_amdgcn_readfirstlane(found[0]);
    if (b < 0) return false;
    const int from = __builtin_amdgcn_readfirstlane(found[1]);
    j = unit - ((from >> 5) + 2 * b);
    s = sequence_from(from, __builtin_amdgcn_readfirstlane(found[2]),
                      __builtin_amdgcn_readfirstlane(found[3]), rows);
  } else {
    s = sequence_of(c, b, rows);
  }
  const int start = s.length - s.n;  // negative with more rows than tokens
  o.b = b;
  o.bn = (start >> 5) + j;
  o.lo = max(start - 32 * o.bn, 0);
  o.hi = min(s.length - 32 * o.bn, 32);
  o.row = s.row0 + 32 * o.bn - start;  // of slot 0
  return o.lo < o.hi;
}

// 8 values of a row
template <bool BF16>
__device__ __forceinline__ void load8(const uint8_t* p, float (&v)[8]) {
  if constexpr (BF16) {
    widen_bf16x8(*reinterpret_cast<const u32x4*>(p), v);
  } else {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(uint8_t* p, const float (&v)[8]) {
  if constexpr (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x2_t t = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
      w[i] = __builtin_bit_cast(uint32_t, t);
    }
    *reinterpret_cast<u32x4*>(p) = u32x4{w[0], w[1], w[2], w[3]};
  } else {
    reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
  }
}

// four codes as they stand in a word, exact in fp32
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float (&v)[4]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 a = FMT == 0 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false)
                           : __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
  const f32x2 b = FMT == 0 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true)
                           : __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}

template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  return fp8_rne_pair<FMT>(a, b) | (fp8_rne_pair<FMT>(c, d) << 16);
}

// 2^(byte - 127), exact, byte 0 .. 254 (0: the subnormal 2^-127)
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return byte ? __uint_as_float(byte << 23) : 0x1p-127f;
}

template <int N>
__device__ __forceinline__ uint32_t workgroup_max(uint32_t m) {
  __shared__ uint32_t part[N];
#pragma unroll
  for (int i = 1; i < 64; i *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, i));
  if constexpr (N > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = part[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = max(m, part[i]);
  }
  return m;
}

// ---------------------------------------------------------------------------------------------
// Writing. A workgroup of dim threads has the keys or the values of one block; a thread 32 of its
// elements: of the keys four runs of 8 in a row, of the values 4 tokens x 8 channels, which make 8
// words of a channel's 4 tokens each: no LDS but for the maximum, whole lines either way.
// 8192 bf16 tokens, 8 heads of 128: 11.0 us in a row (12.0 by the tracer), 4.6 TB/s read and written, what
// a copy reaches (1.5 us more with the rows read after the page was known and each under its condition);
// 64 single tokens: 4.6 us, the chain table - rows - maximum - store.
// ---------------------------------------------------------------------------------------------
template <int D, int FMT, bool BF16, bool CEIL>
__global__ __launch_bounds__(D) void cache_write_kernel(const CacheArgs c, const CacheRows k,
                                                        const CacheRows v) {
  Piece p;
  if (!piece_of(c, blockIdx.x, c.rows, p)) return;
  const int head = blockIdx.y;
  const bool values = blockIdx.z != 0;
  const CacheRows src = values ? v : k;
  const int esize = BF16 ? 2 : 4;
  const uint8_t* rows = static_cast<const uint8_t*>(src.p) + (int64_t)head * src.head * esize;
  const int tid = threadIdx.x;
  // token slot of run i, and its first channel
  auto slot = [&](int i) { return values ? 4 * (tid & 7) + i : (tid + i * D) / (D / 8); };
  auto channel = [&](int i) { return 8 * (values ? tid >> 3 : (tid + i * D) % (D / 8)); };
  // Slots that the call does not fill read a row that it has (a load under a condition would wait for
  // the one before).
  float w[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    load8<BF16>(rows + ((int64_t)(p.row + min(max(slot(i), p.lo), p.hi - 1)) * src.token + channel(i)) * esize,
                w[i]);
  const int64_t block = block_of(c, c.pages, p.b, p.bn, head);  // while the rows are on their way
  if (block < 0) return;
  uint8_t* codes = (values ? c.vq : c.kq) + block * (32 * D);
  uint8_t* scale = (values ? c.vs : c.ks) + block;
  const uint32_t was = p.lo > 0 ? *scale : 0u;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)  // the row read twice changes no maximum
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(w[i][j]));
  m = workgroup_max<D / 64>(m);
  const uint32_t sb = max(scale_byte_fp8<CEIL, FMT>(m), was);
  const bool bad = sb == 0xFFu;  // every code is zero
  // 2^(127 - sb) for what is new; for what is there already 2^(was - sb), at most a flush to zero
  const float up = bad ? 0.0f : __uint_as_float((254u - sb) << 23);
  auto encode = [&](float a, float b, float cc, float d) {
    return bad ? 0u : sb < 254u ? encode4<FMT>(a * up, b * up, cc * up, d * up)
                                : encode4<FMT>(a * 0x1p-127f, b * 0x1p-127f, cc * 0x1p-127f, d * 0x1p-127f);
  };
  if (!values) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = slot(i);
      if (s >= p.lo && s < p.hi)
        *reinterpret_cast<uint2*>(codes + s * D + channel(i)) =
            make_uint2(encode(w[i][0], w[i][1], w[i][2], w[i][3]),
                       encode(w[i][4], w[i][5], w[i][6], w[i][7]));
    }
  } else {
    const int s0 = slot(0), ch = channel(0);
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = encode(w[0][j], w[1][j], w[2][j], w[3][j]);
    if (s0 >= p.lo && s0 + 4 <= p.hi) {
#pragma unroll
      for (int j = 0; j < 8; ++j) *reinterpret_cast<uint32_t*>(codes + (ch + j) * 32 + s0) = o[j];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (s0 + i >= p.lo && s0 + i < p.hi)
#pragma unroll
          for (int j = 0; j < 8; ++j) codes[(ch + j) * 32 + s0 + i] = (uint8_t)(o[j] >> (8 * i));
    }
  }
  if (sb != was || p.lo == 0) {
    if (tid == 0) *scale = (uint8_t)sb;
    // older codes, rounded to the larger scale
    const float again = bad ? 0.0f : ldexpf(1.0f, (int)was - (int)sb);
    auto coarser = [&](uint32_t word) {
      float t[4];
      decode4<FMT>(word, t);
      return bad ? 0u : encode4<FMT>(t[0] * again, t[1] * again, t[2] * again, t[3] * again);
    };
    if (!values) {
      for (int i = tid; i < p.lo * (D / 4); i += D) {
        uint32_t* at = reinterpret_cast<uint32_t*>(codes) + i;
        *at = coarser(*at);
      }
    } else {
      // words of 4 tokens; in the last one the new tokens' bytes are other threads' to write
      const int words = (p.lo + 3) / 4;
      for (int i = tid; i < words * D; i += D) {
        const int q = i / D, ch = i % D, left = min(p.lo - 4 * q, 4);
        uint8_t* at = codes + ch * 32 + 4 * q;
        const uint32_t o = coarser(*reinterpret_cast<const uint32_t*>(at));
        if (left == 4)
          *reinterpret_cast<uint32_t*>(at) = o;
        else
          for (int j = 0; j < left; ++j) at[j] = (uint8_t)(o >> (8 * j));
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Reading back: the same pieces. Positions that have no page (before the first token, too) are zeros.
// 13750 tokens of 8 heads of 128 in bf16: 16.1 us, 5.2 TB/s.
// ---------------------------------------------------------------------------------------------
template <int D, int FMT, bool BF16>
__global__ __launch_bounds__(D) void cache_read_kernel(const CacheArgs c, const CacheRows k,
                                                       const CacheRows v) {
  Piece p;
  if (!piece_of(c, blockIdx.x, c.rows, p)) return;
  const int head = blockIdx.y;
  const bool values = blockIdx.z != 0;
  const int64_t block = block_of(c, c.pages, p.b, p.bn, head);
  const CacheRows dst = values ? v : k;
  const int esize = BF16 ? 2 : 4;
  uint8_t* rows = static_cast<uint8_t*>(const_cast<void*>(dst.p)) + (int64_t)head * dst.head * esize;
  const int tid = threadIdx.x;
  const uint8_t* codes = block < 0 ? nullptr : (values ? c.vq : c.kq) + block * (32 * D);
  const uint32_t sb = block < 0 ? 127u : (values ? c.vs : c.ks)[block];
  const float f = sb == 0xFFu ? __uint_as_float(0x7FC00000u) : scale_of(sb);
  float w[4][8];
  if (block < 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = 0.0f;
  } else if (!values) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint2 q = *reinterpret_cast<const uint2*>(codes + 8 * (tid + i * D));
      float a[4], b[4];
      decode4<FMT>(q.x, a);
      decode4<FMT>(q.y, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[i][j] = a[j] * f;
        w[i][4 + j] = b[j] * f;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float a[4];
      decode4<FMT>(*reinterpret_cast<const uint32_t*>(codes + (8 * (tid >> 3) + j) * 32 + 4 * (tid & 7)), a);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i][j] = a[i] * f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int s = values ? 4 * (tid & 7) + i : (tid + i * D) / (D / 8);
    const int ch = 8 * (values ? tid >> 3 : (tid + i * D) % (D / 8));
    if (s >= p.lo && s < p.hi)
      store8<BF16>(rows + ((int64_t)(p.row + s) * dst.token + ch) * esize, w[i]);
  }
}

// ---------------------------------------------------------------------------------------------
// Attention of a sequence's newest tokens over its cache.
//
// The rows that share a head of the cache, n tokens x `group` query heads, go 16 to a matrix
// product; a wave takes TS tokens of the cache a step:
//   S^T [tokens][rows] = K q^T     a 16 x 16 x 32 product's A row i is a token, its k 8 channels a lane
//   O^T [channels][rows] += V^T P^T   A row i is a channel, k tokens
// Lane (i, g) = (lane & 15, lane >> 4) gets of S^T the column (query row) i and 4 tokens of each of
// its 16-token tiles. Tile t's row i is token (TS / 4) (i / 4) + 4 t + i % 4 of the step, so that lane
// group g has the TS / 4 tokens from (TS / 4) g on: as P^T it is where the second product wants it, and
// the value codes of a channel's same tokens are contiguous. Nothing is transposed or exchanged but
// the maximum of a row, which four lanes hold.
//
// Codes become bf16 with their block's scale in the converter (exact: 4 bits and a power of two).
// q goes in as it is (bf16) or as three bf16 terms that add up to the fp32 value; P as two terms,
// 16 bits, for a bf16 result (the rounding of one, 2^-9, would be felt beside the result's own; with three
// the results are as far from the 64-bit ones, 1.649e-3 of them, and drafts take 5 to 8% longer, single
// tokens up to 2%) and as three for fp32. Sums and the softmax's statistics are fp32, exponentials to the
// base 2.
//
// Work is divided where the lengths are known, on the device, and evenly: a sequence's rows, R = 16 WR
// at a time, are an item, and the steps of all items, one after the other, are cut into as many equal
// parts as there are workgroups (64 sequences of 500 to 16000 tokens, 64 heads over 8 of 128: 171 us, 6.2
// TB/s; with a chunk of a sequence for each workgroup, whatever its length, 25 us more). An item counts
// the whole sequence's steps, though its rows may see fewer: where most of a sequence is new, half of the
// counted steps are empty (4096 tokens of 4096: 1128 us, 244 TFLOP/s; 512 of 2500: 107 us, 351). Short and
// long work and short tables differ, see the constants below. An item in one part is finished there; of the
// others each part goes to the workspace, and a second kernel joins them.
//
// Value codes are read as the product wants them, 4 lanes to a channel's 32 bytes. Key codes are read
// as they lie, 64 lanes x 16 bytes, and ordered through LDS: read in the product's order neighbouring
// lanes have different rows, and each 16 bytes are a line lookup of their own (8 sequences of 4100
// tokens: 24.3 us, 22.3 so; 64 of 8192: 168.7 and 166.4; 256 of 100 to 2000: 118.7 and 111.9).
// ---------------------------------------------------------------------------------------------
constexpr int kWaves = 4;
// Workgroups over all heads: two for each of 256 compute units, which is what their registers allow.
// More of them, or three at a time with fewer registers, read less at once of each page and are slower
// (64 sequences of 8192 tokens: 167 us with 512, 181 with 768 and 175 with 1024).
constexpr int kTarget = 512;
// Long work of single items keeps HBM busier with one workgroup a unit, whose stream is longer, if each
// has kLongSteps steps and more, and its sequences have kLongItem, so that few begin and end (64
// sequences of 500 to 16000 tokens, 64 heads over 8 of 128: 176 us with two, 171 with one; 16 of 16000:
// 86.9 and 84.5; but 256 of 2000: 170 and 180, 4 of 16000: 29.0 and 30.3).
constexpr int kLongSteps = 48, kLongItem = 100;
// Short work: where a wave has up to kShort steps, a workgroup's part is of one item alone, since a
// second segment would cost it the first one's latency again (4 sequences of 4000 tokens, 8 heads of 128:
// 16.8 us cut evenly, 12.9 so; of 200 to 4000: 16.3 and 12.4; one of 8000: 12.3 and 10.6; up to 2 steps
// instead of 4: 4 of 8000 21.5 us for 18.4).
constexpr int kShort = 4;
// Short tables: a workgroup of 8 waves for each item and head, no segments, no second kernel and no
// workspace (8 heads of 128, 16 sequences of 1020 tokens: 13.3 us divided, 11.7; 16 of 50 to 1020: 12.1 and
// 11.0; one of 512: 9.4 and 7.3; one of 1020: 9.5 and 10.5, but 4 us less on the host), as long as the
// workgroups are not very many (256 sequences of 64: 33 and 25); where they are many enough to fill the
// chip, for longer ones too (16 of 1270: 15.1 and 12.8; 4 of 1270: 10.0 and 11.8).
constexpr int kWholeWaves = 8, kWholeItems = 1024;
constexpr int kWholeTokens = 1088, kWholeMost = 1536, kWholeMany = 128;

// 4 channels of an output row: o / sum rounded to the output's type, and once a row its log sum of
// exponentials; a row that sees no token is zeros, -inf
template <bool BF16>
__device__ __forceinline__ void store_row(const AttentionArgs& a, int64_t t, int qhead, int ch,
                                          const f32x4& o, float base, float sum) {
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint8_t* p = static_cast<uint8_t*>(a.out) +
               (t * a.out_token + (int64_t)qhead * a.out_head + ch) * (BF16 ? 2 : 4);
  if constexpr (BF16) {
    const bf16x2_t x = {(__bf16)(o[0] * f), (__bf16)(o[1] * f)};
    const bf16x2_t y = {(__bf16)(o[2] * f), (__bf16)(o[3] * f)};
    *reinterpret_cast<uint2*>(p) =
        make_uint2(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y));
  } else {
    *reinterpret_cast<f32x4*>(p) = f32x4{o[0] * f, o[1] * f, o[2] * f, o[3] * f};
  }
  if (a.lse && ch == 0)
    a.lse[t * a.heads + qhead] =
        sum == 0.0f ? -__builtin_inff() : (base + __builtin_log2f(sum)) * 0.6931471805599453f;
}

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int i = 1; i < 64; i *= 2) v += __shfl_xor(v, i);
  return v;
}

// All steps of all items stand in one line, an item after the other, and each of a head's U workgroups
// has all / U of them, the first all % U one more. A workgroup's part of an item is a segment. Of a
// workgroup's segments only the first and the last one may be part of an item: they have the workspace's
// slots 2 u and 2 u + 1. (The host sees to it that there are fewer than 2^31 steps.)
struct Line {
  int all, at, end;  // steps in all; the workgroup's
  int unit, head;    // the workgroup's
  int units;         // U
  int each, more;    // all / U, all % U
  int part;          // short work: steps of a workgroup, all of one item; else 0
  bool leads;        // `at` is in the workgroup's first segment
  int b, tile;       // the item that step `at` is in: R rows of sequence b from tile * R on
  int first;         // its first step in the line
};

__device__ __forceinline__ int bound_of(const Line& o, int u) { return o.each * u + min(u, o.more); }
// the workgroup that has step x
__device__ __forceinline__ int unit_at(const Line& o, int x) {
  const int longer = o.more * (o.each + 1);
  return x < longer ? (int)((uint32_t)x / (uint32_t)(o.each + 1))
                    : o.more + (int)((uint32_t)(x - longer) / (uint32_t)o.each);
}

template <int R>
__device__ __forceinline__ int items_of(const Sequence& s, int group) {
  return (s.n * group + R - 1) / R;
}
// an item without tokens has a step as well: its rows are written
template <int TS>
__device__ __forceinline__ int steps_of(const CacheArgs& c, const Sequence& s) {
  return max((min(s.length, c.max_tokens) + TS - 1) / TS, 1);
}

// The call's sequences. Up to 64 of them are in the lanes of every wave, and nothing is read again or
// exchanged between waves.
struct Sequences {
  Sequence own;  // of sequence `lane`, where there are 64 at most
  bool few;
  __device__ __forceinline__ Sequence get(const CacheArgs& c, int b) const {
    if (!few) return sequence_of(c, b, c.rows);
    return Sequence{__builtin_amdgcn_readlane(own.row0, b), __builtin_amdgcn_readlane(own.n, b),
                    __builtin_amdgcn_readlane(own.length, b)};
  }
};

// The workgroup's steps, once the line's length is known; false: none. Consecutive workgroups have
// different heads: items of the same sequence and head, which read the same codes, then meet on one XCD
// (4 sequences of 8192 tokens, 16 rows of 64 heads over 8: 56.7 us, 59.5 with a head's in a row). Where
// each sequence and head has one item (SINGLE) its workgroups in a row are 2% faster.
template <bool SINGLE>
__device__ __forceinline__ bool bounds_of(const CacheArgs& c, Line& o, int most) {
  o.units = min(most, o.all);
  if (SINGLE) {
    if (o.all / kLongSteps >= o.units && o.all / kLongItem >= c.seqs) {
      o.units = (o.units + 1) / 2;
    } else {  // a head's workgroups in a row
      const int n = o.unit * c.heads + o.head;
      o.head = (int)((uint32_t)n / (uint32_t)most);
      o.unit = n - o.head * most;
    }
  }
  if (o.unit >= o.units) return false;
  o.each = (int)((uint32_t)o.all / (uint32_t)o.units);
  o.more = o.all - o.each * o.units;
  o.at = bound_of(o, o.unit);
  o.end = bound_of(o, o.unit + 1);
  o.leads = true;
  return true;
}

template <int R, int TS, int WAVES>
__device__ __forceinline__ bool line_of(const CacheArgs& c, const AttentionArgs& a, Line& o,
                                        Sequences& seqs) {
  constexpr bool DIVIDED = WAVES == kWaves;
  const int unit = blockIdx.y, most = gridDim.y;
  o.unit = unit;
  o.head = blockIdx.x;
  o.part = 0;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  auto weight = [&](const Sequence& s) { return DIVIDED ? steps_of<TS>(c, s) : 1; };
  seqs.few = c.seqs <= 64;
  if (!DIVIDED && !c.offsets) {  // as many items for each sequence
    const int each = (a.group + R - 1) / R;
    seqs.few = false;
    o.all = each * c.seqs;
    if (!bounds_of<false>(c, o, most)) return false;
    o.b = unit / each;
    o.tile = unit - o.b * each;
    o.first = unit;
    return true;
  }
  if (seqs.few) {
    const bool is = lane < c.seqs;
    seqs.own = sequence_of(c, is ? lane : 0, c.rows);
    const int n = is ? items_of<R>(seqs.own, a.group) : 0, st = weight(seqs.own);
    auto up_to = [&](int v) {  // the sum of the lanes up to this one
      for (int i = 1; i < c.seqs; i *= 2) {
        const int t = __shfl_up(v, i);
        if (lane >= i) v += t;
      }
      return v;
    };
    for (int k = 1; DIVIDED && k <= kShort;) {
      const int part = k * (WAVES / (R / 16)), parts = (st + part - 1) / part, behind = up_to(n * parts);
      const int total = __builtin_amdgcn_readlane(behind, c.seqs - 1);
      if (total > most) {
        k = total / most >= kShort ? kShort + 1 : max(k + 1, k * total / most);
        continue;
      }
      const uint64_t has = __ballot(is && unit >= behind - n * parts && unit < behind);
      if (has == 0) return false;
      o.b = __builtin_ctzll(has);
      o.part = part;
      const int each = __builtin_amdgcn_readlane(parts, o.b);
      const int at = unit - __builtin_amdgcn_readlane(behind - n * parts, o.b);
      o.tile = (int)((uint32_t)at / (uint32_t)each);
      o.first = 0;
      o.at = (at - o.tile * each) * part;
      o.end = min(o.at + part, __builtin_amdgcn_readlane(st, o.b));
      o.leads = true;
      return true;
    }
    const int end = up_to(n * st);
    o.all = __builtin_amdgcn_readlane(end, c.seqs - 1);
    if (o.all == 0 || !bounds_of<DIVIDED && R == 16>(c, o, most)) return false;
    const int begin = end - n * st;
    const uint64_t has = __ballot(is && o.at >= begin && o.at < end);
    if (has == 0) return false;  // offsets that fall may give more than 2^31 steps
    o.b = __builtin_ctzll(has);
    const int first = __builtin_amdgcn_readlane(begin, o.b);
    const int steps = __builtin_amdgcn_readlane(st, o.b);
    o.tile = (int)((uint32_t)(o.at - first) / (uint32_t)steps);
    o.first = first + o.tile * steps;
    return true;
  }
  __shared__ int sums[WAVES];
  __shared__ unsigned long long got;  // the sequence and its first step
  constexpr unsigned long long none = ~0ull;
  int all = 0;
  for (int b = tid; b < c.seqs; b += 64 * WAVES) {
    const Sequence s = sequence_of(c, b, c.rows);
    all += items_of<R>(s, a.group) * weight(s);
  }
  all = wave_sum(all);
  if (lane == 0) sums[wave] = all;
  if (tid == 0) got = none;
  __syncthreads();
  o.all = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) o.all += sums[i];
  if (o.all == 0 || !bounds_of<DIVIDED && R == 16>(c, o, most)) return false;
  int before = 0;
  for (int b0 = 0; b0 < c.seqs; b0 += 64 * WAVES) {  // the same turns in every wave
    const int b = b0 + tid;
    int n = 0, st = 0;
    if (b < c.seqs) {
      const Sequence s = sequence_of(c, b, c.rows);
      n = items_of<R>(s, a.group);
      st = weight(s);
    }
    int end = n * st;
#pragma unroll
    for (int i = 1; i < 64; i *= 2) {
      const int t = __shfl_up(end, i);
      if (lane >= i) end += t;
    }
    __syncthreads();
    if (lane == 63) sums[wave] = end;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      if (i < wave) end += sums[i];
      total += sums[i];
    }
    end += before;
    const int begin = end - n * st;
    // Offsets that fall may give so many steps that the sums wrap and several sequences have this one:
    // the first of them, with its own start (its steps are fewer than 2^31, so the tile is one of it).
    if (o.at >= begin && o.at < end) atomicMin(&got, (unsigned long long)b << 32 | (uint32_t)begin);
    before += total;
    __syncthreads();
    if (got != none) break;
  }
  if (got == none) return false;
  o.b = __builtin_amdgcn_readfirstlane((int)(got >> 32));
  const int first = __builtin_amdgcn_readfirstlane((int)(uint32_t)got);
  const int st = weight(sequence_of(c, o.b, c.rows));
  o.tile = (int)((uint32_t)(o.at - first) / (uint32_t)st);
  o.first = first + o.tile * st;
  return true;
}

// 8 codes as bf16 values times the scale
template <int FMT>
__device__ __forceinline__ bf16x8_t codes_of(uint32_t lo, uint32_t hi, float f) {
  if constexpr (FMT == 0) {
    const u32x4 o = {
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, true)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, true))};
    return __builtin_bit_cast(bf16x8_t, o);
  } else {
    const u32x4 o = {
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, f, true)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, f, true))};
    return __builtin_bit_cast(bf16x8_t, o);
  }
}

__device__ __forceinline__ f32x4 mfma(bf16x8_t a, bf16x8_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// the larger of a row's values, which lanes i, i + 16, i + 32 and i + 48 hold
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// A load of what only this wave reads (STREAM): past the caches' order of replacement.
template <bool STREAM, typename T>
__device__ __forceinline__ T load_codes(const uint8_t* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
  return *reinterpret_cast<const T*>(p);
}

// The codes of a step's tokens in a lane, and its block's scale (NB == 1: the lanes have one block)
template <int D, int TS>
struct Keys {
  u32x4 w[TS / 16][D / 64];  // as they lie in the cache
  uint32_t scale;
};
template <int D, int TS>
struct Values {
  uint32_t w[D / 16][TS / 16];
  uint32_t scale;
};
// the step's blocks, of which `has` are in the cache (the others stand for block 0)
template <int NB>
struct Blocks {
  int64_t at[NB];
  bool has[NB];
};

template <int D, int TS, int WAVES>
struct AttentionShared {
  // rows of D code bytes; 16 bytes between them and 16 more after 16 rows spread them over the banks
  // (without the latter 25.9 us for 24.6, 20 sequences of 500 to 2000 tokens, fp32, 4 heads of 192)
  static constexpr int PITCH = D + 16, KEYS = TS * PITCH + TS;
  union {
    float part[WAVES][16][D + 4];
    uint8_t keys[WAVES][KEYS];
  };
  float stat[WAVES][16][2];
  static __device__ __forceinline__ int at(int row) { return row * PITCH + (row >> 4) * 16; }
};

// a wave's LDS accesses complete in order; the compiler keeps them so
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One segment: the steps of an item that the workgroup has
template <int D, int FMT, bool BF16, int WR, int TS, int WAVES>
__device__ __forceinline__ void attend(const CacheArgs& c, const AttentionArgs& a,
                                       const int32_t* __restrict__ pages, const Line& line,
                                       const Sequence& s, AttentionShared<D, TS, WAVES>& sh) {
  constexpr int R = 16 * WR, TW = WAVES / WR;  // rows a workgroup; waves that share a row's tokens
  constexpr int NQ = BF16 ? 1 : 3, NP = BF16 ? 2 : 3, KT = TS / 16, NB = TS / 32, PER = TS / 4;
  const int head = line.head, unit = line.unit;
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wr = wave % WR, wt = wave / WR;
  const int all_steps = steps_of<TS>(c, s);
  constexpr bool WHOLE = WAVES != kWaves;
  const int from = WHOLE ? 0 : line.at - line.first;
  const int to = WHOLE ? all_steps : min(line.end - line.first, all_steps);
  // the item's segments are those of units first_unit .. last_unit
  const bool shorts = !WHOLE && line.part > 0;
  const int first_unit = from == 0 ? unit : shorts ? unit - from / line.part : unit_at(line, line.first);
  const int last_unit = to == all_steps ? unit
                        : shorts        ? first_unit + (all_steps - 1) / line.part
                                        : unit_at(line, line.first + all_steps - 1);
  const int row0 = line.tile * R;
  const int rows = s.n * a.group;      // of this sequence and head
  const int row = row0 + 16 * wr + i;  // this lane's
  const int token = min(row, rows - 1) / a.group, qhead = head * a.group + min(row, rows - 1) % a.group;
  // how many tokens a row sees; rows past the end see what the last one does and are not stored
  const int seen = min(s.length - s.n + token + 1, c.max_tokens);
  const int wg_last = (min(row0 + R, rows) - 1) / a.group;  // the last token of the unit's rows
  const int most = min(s.length - s.n + wg_last + 1, c.max_tokens);
  const int first_token = min(row0 + 16 * wr, rows - 1) / a.group;
  const int least = min(s.length - s.n + first_token + 1, c.max_tokens);  // of this wave's rows
  const int end = row0 + 16 * wr < rows  // a wave may have no rows
                      ? min(to, (max(most, 0) + TS - 1) / TS) : 0;

  bf16x8_t q[NQ][D / 32];
  {
    const uint8_t* p = static_cast<const uint8_t*>(a.q) +
                       ((int64_t)(s.row0 + token) * a.q_token + (int64_t)qhead * a.q_head) * (BF16 ? 2 : 4);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {  // channels 64 (j / 2) + 16 g + 8 (j % 2) ..
      const int ch = 64 * (j / 2) + 16 * g + 8 * (j % 2);
      if constexpr (BF16) {
        q[0][j] = *reinterpret_cast<const bf16x8_t*>(p + ch * 2);
      } else {
        float t[8];
        load8<false>(p + ch * 4, t);
        uint32_t o[4][3];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_pair<3>(t[2 * e], t[2 * e + 1], o[e]);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
          q[n][j] = __builtin_bit_cast(bf16x8_t, u32x4{o[0][n], o[1][n], o[2][n], o[3][n]});
      }
    }
  }

  f32x4 acc[D / 16];
#pragma unroll
  for (int d = 0; d < D / 16; ++d) acc[d] = f32x4{0, 0, 0, 0};
  float m = -__builtin_inff(), l = 0.0f;

  // the page numbers of a step's blocks; past the end those of the table's first page
  const int32_t* table = pages + (int64_t)line.b * c.table_width;
  auto look = [&](int step, int (&page)[NB]) {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int slot = slot_of(c, NB * step + n);
      page[n] = table[step < end && slot < c.table_width ? slot : 0];
    }
  };
  auto find = [&](int step, const int (&page)[NB]) {
    Blocks<NB> o;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int bn = NB * step + n, slot = slot_of(c, bn);
      o.has[n] = step < end && 32 * bn < most && page[n] >= 0 && page[n] < c.n_pages;
      const int64_t at = ((int64_t)page[n] * c.heads + head) * c.page_blocks + (bn - slot * c.page_blocks);
      o.at[n] = o.has[n] ? at : 0;
    }
    return o;
  };
  auto load_keys = [&](const Blocks<NB>& b, Keys<D, TS>& o) {
    const int64_t at = NB == 1 ? b.at[0] : i >= 8 ? b.at[NB - 1] : b.at[0];
    o.scale = c.ks[at];
    // 64 lanes x 16 bytes in a row each: D / 32 of these loads are a block's keys
#pragma unroll
    for (int n = 0; n < KT * (D / 64); ++n) {
      const int64_t from = b.at[n / (D / 32)] * (32 * D) + (n % (D / 32)) * 1024 + lane * 16;
      o.w[n / (D / 64)][n % (D / 64)] = load_codes<WR == 1, u32x4>(c.kq + from);
    }
  };
  auto load_values = [&](const Blocks<NB>& b, Values<D, TS>& o) {
    const int64_t at = NB == 1 ? b.at[0] : g >= 2 ? b.at[NB - 1] : b.at[0];
    o.scale = c.vs[at];
    const uint8_t* p = c.vq + at * (32 * D) + i * 32 + PER * (g & (NB == 1 ? 3 : 1));
    typedef uint32_t word __attribute__((ext_vector_type(TS / 16)));
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      const word w = load_codes<WR == 1, word>(p + d * 512);
#pragma unroll
      for (int t = 0; t < KT; ++t) o.w[d][t] = w[t];
    }
  };

  int step = from + wt;
  Keys<D, TS> k;
  Values<D, TS> v;
  Blocks<NB> here, next;
  if (step < end) {
    int page[NB], page2[NB];
    look(step, page);
    look(step + TW, page2);
    here = find(step, page);
    load_keys(here, k);
    load_values(here, v);
    next = find(step + TW, page2);
  }
  // The next step's keys are on their way while this one's softmax and values are worked on, and its
  // values during its scores, in the registers that have just become free.
  auto take = [&](auto follows) {
    constexpr bool more = decltype(follows)::value;
    int page[NB];
    if constexpr (more) look(step + 2 * TW, page);
    // the keys into the order of the product, in LDS of the wave's own
    uint8_t* keys = sh.keys[wave];
    wave_order();
#pragma unroll
    for (int n = 0; n < KT * (D / 64); ++n) {
      const int byte = n * 1024 + lane * 16;
      *reinterpret_cast<u32x4*>(keys + sh.at(byte / D) + byte % D) = k.w[n / (D / 64)][n % (D / 64)];
    }
    wave_order();
    const uint32_t kscale = k.scale;
    if constexpr (more) load_keys(next, k);
    f32x4 sc[KT];
    const bool nan_k = kscale == 0xFFu;
    const float kf = nan_k ? 1.0f : scale_of(kscale);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      sc[t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(
            keys + sh.at(PER * (i >> 2) + 4 * t + (i & 3)) + 64 * j + 16 * g);
        const bf16x8_t k0 = codes_of<FMT>(w[0], w[1], kf);
        const bf16x8_t k1 = codes_of<FMT>(w[2], w[3], kf);
#pragma unroll
        for (int n = NQ - 1; n >= 0; --n) {
          sc[t] = mfma(k0, q[n][2 * j], sc[t]);
          sc[t] = mfma(k1, q[n][2 * j + 1], sc[t]);
        }
      }
    }
    bool whole = (step + 1) * TS <= least;
#pragma unroll
    for (int n = 0; n < NB; ++n) whole = whole && here.has[n];
    const bool nan_v = v.scale == 0xFFu;
    const float vf = nan_v ? 1.0f : scale_of(v.scale);
    // a block whose maximum was not finite: what sees it is NaN, and its codes are zero
    const bool strange = __any(nan_k || nan_v);
    float p[KT][4];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) p[t][r] = sc[t][r] * a.scale_log2;
    bool lost = false;  // this lane's tokens have no values
    int mine = PER;     // of this lane's tokens, those that its row sees
    if (!whole || strange) {
      // tokens PER g .. of the step are this lane's, in block g / 2 of two
      const bool has = NB == 1 ? here.has[0] : g >= 2 ? here.has[NB - 1] : here.has[0];
      const int at = step * TS + PER * g;
      mine = has ? min(seen - at, PER) : 0;
      const int held = has ? min(most - at, PER) : 0;  // that any row sees
      // the scales of the block that this lane's scores come from
      const uint32_t kb = NB == 1 ? kscale : (uint32_t)__shfl((int)kscale, g >= 2 ? 8 : 0);
      const bool nan = kb == 0xFFu;
      lost = nan_v;
#pragma unroll
      for (int t = 0; t < KT; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          p[t][r] = 4 * t + r < mine ? nan ? __builtin_nanf("") : p[t][r] : -__builtin_inff();
        const int left = nan_v ? 0 : min(max(held - 4 * t, 0), 4);
        const uint32_t keep = left == 4 ? 0xFFFFFFFFu : (1u << (8 * left)) - 1u;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) v.w[d][t] &= keep;
      }
    }
    float top = p[0][0];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) top = fmaxf(top, p[t][r]);
    top = row_max(top);
    if (__any(top > m)) {
      const float next = fmaxf(m, top);
      const float f = next == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - next);
      l *= f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[d][r] *= f;
      m = next;
    }
    const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        p[t][r] = __builtin_amdgcn_exp2f(p[t][r] - base);
        l += p[t][r];
      }
    if (strange) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (lost && 4 * t + r < mine) p[t][r] = __builtin_nanf("");
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {  // 8 tokens a lane: tiles 2b and 2b + 1
      uint32_t w[4][NP];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        split_pair<NP>(p[2 * b + e / 2][2 * (e % 2)], p[2 * b + e / 2][2 * (e % 2) + 1], w[e]);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        const bf16x8_t x = codes_of<FMT>(v.w[d][2 * b], v.w[d][2 * b + 1], vf);
#pragma unroll
        for (int n = NP - 1; n >= 0; --n)
          acc[d] = mfma(x, __builtin_bit_cast(bf16x8_t, u32x4{w[0][n], w[1][n], w[2][n], w[3][n]}), acc[d]);
      }
    }
    if constexpr (more) {
      load_values(next, v);
      here = next;
      next = find(step + 2 * TW, page);
    }
  };
  for (; step + TW < end; step += TW) take(std::true_type());
  if (step < end) take(std::false_type());

  __syncthreads();  // keys and parts share LDS
  // the waves' parts of a row, joined in the waves' order
  l = row_sum(l);
  if (l != l) m = 0.0f;  // a NaN counts, whatever the maximum of the others
  if (g == 0) {
    sh.stat[wave][i][0] = m;
    sh.stat[wave][i][1] = l;
  }
#pragma unroll
  for (int d = 0; d < D / 16; ++d)
    *reinterpret_cast<f32x4*>(&sh.part[wave][i][16 * d + 4 * g]) = acc[d];
  __syncthreads();
  for (int e = tid; e < R * (D / 4); e += 64 * WAVES) {
    const int r = e / (D / 4), ch = 4 * (e % (D / 4)), at = row0 + r;
    if (at >= rows) break;
    const int w0 = r / 16, ri = r % 16;
    float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
    for (int w = 0; w < TW; ++w) top = fmaxf(top, sh.stat[w0 + w * WR][ri][0]);
    const float base = top == -__builtin_inff() ? 0.0f : top;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < TW; ++w) {
      const float f = __builtin_amdgcn_exp2f(sh.stat[w0 + w * WR][ri][0] - base);
      sum += sh.stat[w0 + w * WR][ri][1] * f;
      const f32x4 t = *reinterpret_cast<const f32x4*>(&sh.part[w0 + w * WR][ri][ch]);
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] += t[x] * f;
    }
    const int part = 2 * unit + (line.leads ? 0 : 1);
    const int64_t slot = ((int64_t)part * c.heads + head) * R + r;
    if (first_unit == last_unit) {
      store_row<BF16>(a, (int64_t)s.row0 + at / a.group, head * a.group + at % a.group, ch, o, base, sum);
    } else {
      *reinterpret_cast<f32x4*>(a.part + slot * D + ch) = o;
      if (ch == 0) {
        a.stat[2 * slot] = top;
        a.stat[2 * slot + 1] = sum;
      }
    }
  }
  if (!WHOLE && a.where && from == 0 && head == 0 && tid < R && row0 + tid < rows) {
    const int at = row0 + tid;
    const int first = 2 * unit + (line.leads ? 0 : 1);
    a.where[(int64_t)s.row0 * a.group + at] = make_int4(first, last_unit - first_unit + 1, tid, 0);
  }
}

template <int D, int FMT, bool BF16, int WR, int TS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void cache_attention_kernel(
    const CacheArgs c, const AttentionArgs a, const int32_t* __restrict__ pages) {
  __shared__ __attribute__((aligned(16))) AttentionShared<D, TS, WAVES> sh;
  Line line;
  Sequences seqs;
  if (!line_of<16 * WR, TS, WAVES>(c, a, line, seqs)) return;
  for (;;) {
    const Sequence s = seqs.get(c, line.b);
    attend<D, FMT, BF16, WR, TS, WAVES>(c, a, pages, line, s, sh);
    if (WAVES != kWaves) return;  // the item whole
    line.at = line.first + steps_of<TS>(c, s);
    if (line.at >= line.end) return;
    line.first = line.at;
    line.leads = false;
    if (++line.tile * 16 * WR >= s.n * a.group) {
      line.tile = 0;
      do {
        if (++line.b >= c.seqs) return;
      } while (seqs.get(c, line.b).n == 0);
    }
    __syncthreads();  // what the waves read of sh is written again
  }
}

// The segments of a row joined. THREADS for each token and query head: 256 where the rows are few and
// may have many segments, a wave where there are many rows. A thread has 4 channels; groups of D / 4
// threads take every GROUPS-th segment.
template <int D, bool BF16, int THREADS>
__global__ __launch_bounds__(256) void cache_attention_join_kernel(const CacheArgs c,
                                                                   const AttentionArgs a, int R) {
  constexpr int PER = D / 4, GROUPS = THREADS / PER, ROWS = 256 / THREADS;
  __shared__ __attribute__((aligned(16))) float sums[ROWS][GROUPS][D];
  __shared__ float tops[ROWS][GROUPS], all[ROWS][GROUPS];
  const int which = threadIdx.x / THREADS, tid = threadIdx.x % THREADS;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * ROWS + which;
  const int t = (int)(row / a.heads), qhead = (int)(row - (int64_t)t * a.heads), head = qhead / a.group;
  bool is = t < c.rows;
  if (is && c.offsets) is = t >= c.offsets[0] && t < c.offsets[c.seqs];
  int4 w = make_int4(0, 0, 0, 0);
  if (is) w = a.where[(int64_t)t * a.group + qhead - head * a.group];
  // one part: written already; and tables that are none (offsets that fall) end here
  if (w.y <= 1 || w.x < 0 || w.z < 0 || w.z >= R || (int64_t)w.x / 2 + w.y > a.slots / 2) is = false;
  const int group = tid / PER, ch = 4 * (tid % PER);
  if (is && group < GROUPS) {
    f32x4 o = {0, 0, 0, 0};
    float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll 4
    for (int k = group; k < w.y; k += GROUPS) {
      const int slot = k == 0 ? w.x : 2 * (w.x / 2 + k);
      const int64_t s = ((int64_t)slot * c.heads + head) * R + w.z;
      const float m = a.stat[2 * s], l = a.stat[2 * s + 1];
      const f32x4 v = *reinterpret_cast<const f32x4*>(a.part + s * D + ch);
      const float next = fmaxf(top, m), base = next == -__builtin_inff() ? 0.0f : next;
      const float f = __builtin_amdgcn_exp2f(top - base), h = __builtin_amdgcn_exp2f(m - base);
      sum = sum * f + l * h;
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] = o[x] * f + v[x] * h;
      top = next;
    }
    *reinterpret_cast<f32x4*>(&sums[which][group][ch]) = o;
    if (ch == 0) {
      tops[which][group] = top;
      all[which][group] = sum;
    }
  }
  __syncthreads();
  if (is && tid < PER) {
    float top = tops[which][0];
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) top = fmaxf(top, tops[which][k]);
    const float base = top == -__builtin_inff() ? 0.0f : top;
    f32x4 o = {0, 0, 0, 0};
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      const float f = __builtin_amdgcn_exp2f(tops[which][k] - base);
      sum += all[which][k] * f;
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] += sums[which][k][4 * tid + x] * f;
    }
    store_row<BF16>(a, t, qhead, 4 * tid, o, base, sum);
  }
}

template <int D, int FMT, bool BF16>
hipError_t launch_write(const CacheArgs& c, const CacheRows& k, const CacheRows& v, bool ceil,
                        int64_t units, void* stream) {
  const dim3 grid((unsigned)units, (unsigned)c.heads, 2);
  if (ceil)
    hipLaunchKernelGGL((cache_write_kernel<D, FMT, BF16, true>), grid, dim3(D), 0,
                       (hipStream_t)stream, c, k, v);
  else
    hipLaunchKernelGGL((cache_write_kernel<D, FMT, BF16, false>), grid, dim3(D), 0,
                       (hipStream_t)stream, c, k, v);
  return hipGetLastError();
}

template <int D, int FMT, bool BF16>
hipError_t launch_read(const CacheArgs& c, const CacheRows& k, const CacheRows& v, int64_t units,
                       void* stream) {
  hipLaunchKernelGGL((cache_read_kernel<D, FMT, BF16>), dim3((unsigned)units, (unsigned)c.heads, 2),
                     dim3(D), 0, (hipStream_t)stream, c, k, v);
  return hipGetLastError();
}

// dim, format and type of a call as template arguments
template <template <int, int, bool> class F, int D, typename... A>
hipError_t pick_type(const CacheArgs& c, bool bf16, A&&... args) {
  if (c.fmt == 0) return bf16 ? F<D, 0, true>::run(c, args...) : F<D, 0, false>::run(c, args...);
  return bf16 ? F<D, 1, true>::run(c, args...) : F<D, 1, false>::run(c, args...);
}
template <template <int, int, bool> class F, typename... A>
hipError_t pick(const CacheArgs& c, bool bf16, A&&... args) {
  switch (c.dim) {
    case 64: return pick_type<F, 64>(c, bf16, args...);
    case 128: return pick_type<F, 128>(c, bf16, args...);
    case 192: return pick_type<F, 192>(c, bf16, args...);
    default: return pick_type<F, 256>(c, bf16, args...);
  }
}

template <int D, int FMT, bool BF16>
struct Write {
  static hipError_t run(const CacheArgs& c, const CacheRows& k, const CacheRows& v, bool ceil,
                        int64_t units, void* stream) {
    return launch_write<D, FMT, BF16>(c, k, v, ceil, units, stream);
  }
};
template <int D, int FMT, bool BF16>
struct Read {
  static hipError_t run(const CacheArgs& c, const CacheRows& k, const CacheRows& v, int64_t units,
                        void* stream) {
    return launch_read<D, FMT, BF16>(c, k, v, units, stream);
  }
};

// units of the calls' rows, see piece_of
int64_t pieces(const CacheArgs& c) {
  return c.offsets ? (int64_t)c.rows / 32 + 2 * (int64_t)c.seqs : c.seqs;
}

// tokens of a step: wider heads take fewer, for their registers (fp32 has too many all the same: 64
// sequences of 3000 to 5000 tokens, 16 heads over 4: dim 128 56 us; 192, 7 registers spilled, 90; 256, 71
// of them, 183)
constexpr int step_tokens(int dim) { return dim <= 128 ? 64 : 32; }

struct AttentionPlan {
  // Row tiles of a workgroup, from the average of the sequences' rows, which the host knows: an uneven call
  // is slower than its parts (512 tokens of 2500 and 63 single ones of 8000: 408 us, 107 and 161 apart).
  int wr;
  int64_t units;   // workgroups for each head
  int64_t slots;   // of the workspace, two for each workgroup
  bool whole;      // a workgroup for each item and head
  bool join;
};

AttentionPlan plan_attention(const CacheArgs& c, const AttentionArgs& a) {
  AttentionPlan p;
  const int64_t rows = (int64_t)c.rows * a.group;
  const int64_t each = c.offsets ? (rows + c.seqs - 1) / c.seqs : a.group;
  p.wr = each <= 16 ? 1 : each <= 32 ? 2 : 4;
  const int64_t items = rows / (16 * p.wr) + c.seqs;
  const int64_t most = (c.max_tokens + step_tokens(c.dim) - 1) / step_tokens(c.dim);
  const int64_t steps = most > 0 ? most : 1;
  const int64_t workgroups = items * c.heads;
  p.whole = p.wr == 1 && workgroups <= kWholeItems &&
            c.max_tokens <= (workgroups < kWholeMany ? kWholeTokens : kWholeMost);
  p.join = !p.whole && steps > 1;
  p.units = (kTarget + c.heads - 1) / c.heads;
  if (p.whole) p.units = items;
  else if (items * steps < p.units) p.units = items * steps;
  p.slots = 2 * p.units;
  return p;
}

template <int D, int FMT, bool BF16>
struct Attention {
  template <int WR, int WAVES>
  static void main(const CacheArgs& c, const AttentionArgs& a, const AttentionPlan& p) {
    hipLaunchKernelGGL((cache_attention_kernel<D, FMT, BF16, WR, step_tokens(D), WAVES>),
                       dim3((unsigned)c.heads, (unsigned)p.units), dim3(64 * WAVES), 0,
                       (hipStream_t)a.stream, c, a, c.pages);
  }
  static hipError_t run(const CacheArgs& c, const AttentionArgs& a, const AttentionPlan& p) {
    if (p.whole) main<1, kWholeWaves>(c, a, p);
    else if (p.wr == 1) main<1, kWaves>(c, a, p);
    else if (p.wr == 2) main<2, kWaves>(c, a, p);
    else main<4, kWaves>(c, a, p);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || !p.join) return e;
    const int64_t rows = (int64_t)c.rows * a.heads;
    // 4096 rows: 4.8 us with a wave each, 6.0 with a workgroup; 32 rows of 32 parts: 5.6 and 4.3
    if (rows < 2048) {
      hipLaunchKernelGGL((cache_attention_join_kernel<D, BF16, 256>), dim3((unsigned)rows), dim3(256), 0,
                         (hipStream_t)a.stream, c, a, 16 * p.wr);
    } else {
      // up to 2^28 workgroups: a dimension of a grid holds fewer than 2^32 threads
      const int64_t workgroups = (rows + 3) / 4, most = (int64_t)1 << 22;
      const int64_t x = workgroups < most ? workgroups : most;
      hipLaunchKernelGGL((cache_attention_join_kernel<D, BF16, 64>),
                         dim3((unsigned)x, (unsigned)((workgroups + x - 1) / x)), dim3(256), 0,
                         (hipStream_t)a.stream, c, a, 16 * p.wr);
    }
    return hipGetLastError();
  }
};

// steps of all items, at most
int64_t all_steps(const CacheArgs& c, const AttentionArgs& a) {
  const AttentionPlan p = plan_attention(c, a);
  const int ts = step_tokens(c.dim);
  return ((int64_t)c.rows * a.group / (16 * p.wr) + c.seqs) * ((int64_t)c.max_tokens / ts + 1);
}

int64_t part_floats(const CacheArgs& c, const AttentionPlan& p) {
  return p.join ? p.slots * c.heads * 16 * p.wr : 0;
}

}  // namespace

hipError_t mx_launch_cache_write(const CacheArgs& c, const CacheRows& k, const CacheRows& v,
                                 bool bf16, bool ceil, void* stream) {
  return pick<Write>(c, bf16, k, v, ceil, pieces(c), stream);
}

hipError_t mx_launch_cache_read(const CacheArgs& c, const CacheRows& k, const CacheRows& v,
                                bool bf16, void* stream) {
  return pick<Read>(c, bf16, k, v, pieces(c), stream);
}

bool mx_attention_fits(const CacheArgs& c, const AttentionArgs& a) {
  return all_steps(c, a) < ((int64_t)1 << 31);
}

// [where: 16 bytes a row][part: D floats][stat: 2 floats] for each chunk's row
int64_t mx_attention_workspace_bytes(const CacheArgs& c, const AttentionArgs& a) {
  const AttentionPlan p = plan_attention(c, a);
  return p.join ? 16 * (int64_t)c.rows * a.group + part_floats(c, p) * (c.dim + 2) * 4 : 0;
}

hipError_t mx_launch_cache_attention(const CacheArgs& c, AttentionArgs a, void* workspace) {
  const AttentionPlan p = plan_attention(c, a);
  a.slots = p.slots;
  if (p.join) {
    a.where = static_cast<int4*>(workspace);
    a.part = reinterpret_cast<float*>(a.where + (int64_t)c.rows * a.group);
    a.stat = a.part + part_floats(c, p) * c.dim;
  }
  return pick<Attention>(c, a.bf16, a, p);
}
