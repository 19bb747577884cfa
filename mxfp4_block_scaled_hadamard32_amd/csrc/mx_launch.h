// mx_launch.h — internal interface between the C ABI layer (mx_api.hip) and the kernel
// launchers (quant.hip, gemm.hip, norm.hip, gemv.hip, cache.hip, lora.hip). Arguments are already validated when these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct QuantArgs {
  const void* x;
  bool bf16;
  int64_t rows, cols, ld;
  int axis;          // 1D only
  bool ceil, sr, hadamard;
  uint32_t sign_mask;
  uint64_t seed;
  uint8_t* codes;    // axis 1 / 2-D: [rows][cols/2];  axis 0: [cols][rows/2]
  uint8_t* scales;
  uint8_t* codes_t;  // 2-D only, nullable
  uint8_t* scales_t; // 2-D only, nullable
  void* stream;
};

hipError_t mx_launch_quantize(const QuantArgs& a);
hipError_t mx_launch_quantize_2d(const QuantArgs& a);
// MXFP8 1x32 quantize (fmt 0 = E4M3, 1 = E5M2): codes one byte per element,
// axis 1: [rows][cols], axis 0: [cols][rows]; scales as for MXFP4
hipError_t mx_launch_quantize_fp8(const QuantArgs& a, int fmt);
// B x B tiles (block 8, 32 or 64; rows and cols multiples of max(block, 32)); for 64 the scales
// are in the GEMM layout [rows/64][cols/32] / [cols/64][rows/32] (each byte twice)
hipError_t mx_launch_quantize_2d_blocks(const QuantArgs& a, int block);
// map[r][c] = scale byte of the row block of (r, c) minus that of its column block (int8,
// saturated; -128 for a non-finite block); rows, cols multiples of 32
hipError_t mx_launch_scale_mismatch(const void* x, bool bf16, int64_t rows, int64_t cols,
                                    int64_t ld, bool ceil, int8_t* map, void* stream);
hipError_t mx_launch_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int64_t cols, int block_rows, int inv_had, uint32_t sign_mask,
                                float* out, void* stream);

// C[m][n] = 2^alpha * sum_k A[m][k] * B[n][k]; A [M][K/2], B [N][K/2] packed E2M1, scales
// [M/ga][K/32] and [N/gb][K/32].
struct GemmArgs {
  const uint8_t* a;
  const uint8_t* as;
  int ga;
  const uint8_t* b;
  const uint8_t* bs;
  int gb;
  int64_t M, N, K;
  int alpha;
  bool out_bf16;
  void* c;
  int64_t ldc;
  void* stream;
};

hipError_t mx_launch_gemm(const GemmArgs& g);

// Epilogue quantization of C along its rows (1x32 blocks along N), instead of storing C:
// codes [M][N/2], scales [M][N/32]; the random-field index of C[m][n] is m * N + n.
struct GemmQuantOut {
  uint8_t* codes;
  uint8_t* scales;
  bool hadamard, sr, ceil;
  uint32_t sign_mask;
  uint64_t seed;
};

// K must be a multiple of 128 (the streaming kernels); returns hipErrorInvalidValue otherwise.
hipError_t mx_launch_gemm_quant(const GemmArgs& g, const GemmQuantOut& q);

// MXFP8 GEMM: A [M][K], B [N][K] one code byte per element (afmt / bfmt: 0 = E4M3, 1 = E5M2),
// scales [M][K/32] and [N][K/32] (ga = gb = 1). K must be a positive multiple of 128.
hipError_t mx_launch_gemm_fp8(const GemmArgs& g, int afmt, int bfmt);

// RMS norm of [rows][cols] (cols a positive multiple of 32, at most kNormMaxCols): s = x
// (+ residual), outputs each optional: the rounded sum, y, rstd, and codes with scales of fmt
// 0 none, 1 E2M1, 2 E4M3, 3 E5M2.
constexpr int64_t kNormMaxCols = 32768;
struct NormArgs {
  const void* x;
  const void* residual;
  const void* gamma;
  void* sum;
  void* y;
  float* rstd;
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows, cols, ldx, ldr, lds, ldy;
  uint64_t seed;
  double inv_cols;  // set by the launcher
  float eps;
  uint32_t sign_mask;
  int fmt;
  bool bf16, gamma_bf16, ceil, sr, hadamard;
  void* stream;
};
hipError_t mx_launch_rmsnorm(const NormArgs& a);

// Its backward pass. partial: at least mx_norm_backward_blocks(rows, cols) * cols floats (the most
// that either type uses; 0 for small tensors), NULL without dgamma.
struct NormBackwardArgs {
  const void* dy;
  const void* dsum;
  const void* s;
  const void* gamma;
  const float* rstd;
  void* dx;
  float* dgamma;
  float* partial;
  int64_t rows, cols, lddy, ldds, lds, lddx;
  bool bf16, gamma_bf16;
  void* stream;
  float inv_cols;  // set by the launcher, as row_blocks
  int row_blocks;
};
int64_t mx_norm_backward_blocks(int64_t rows, int64_t cols);
hipError_t mx_launch_rmsnorm_backward(const NormBackwardArgs& a);

// y[t][n] = 2^alpha * sum_k x[t][k] * W[n][k]; x bf16 or fp32, W packed E2M1 with scales
// [N/gw][K/32]. The limits keep every shape's grid (16 tokens by 16 rows a workgroup at least)
// within 2^22 x 2^15 workgroups.
constexpr int64_t kGemvMaxTokens = (int64_t)1 << 19, kGemvMaxRows = (int64_t)1 << 26;
struct GemvArgs {
  const void* x;
  const uint8_t* w;
  const uint8_t* ws;
  void* y;
  int64_t T, N, K, ldx, ldy;
  int gw, alpha;
  uint32_t sign_mask;
  bool bf16, hadamard, out_bf16;
  void* stream;
  float* part;  // mx_gemv_workspace_bytes of workspace where that is not 0, or NULL
};
int64_t mx_gemv_workspace_bytes(int64_t T, int64_t N, int64_t K, bool bf16, bool hadamard,
                                bool out_bf16);
hipError_t mx_launch_gemv(const GemvArgs& a);

// A paged cache of 8-bit keys and values (mx_cache of mx.h) and the rows of one call on it. Row r of
// the call belongs to sequence r, or with offsets rows offsets[b] .. offsets[b + 1] to sequence b.
struct CacheArgs {
  uint8_t* kq;
  uint8_t* ks;
  uint8_t* vq;
  uint8_t* vs;
  const int32_t* pages;    // [seqs][table_width]
  const int32_t* lengths;  // [seqs]
  const int32_t* offsets;  // [seqs + 1] or NULL
  int n_pages, seqs, table_width, heads, dim, rows;
  int page_blocks;         // page size / 32, at most kCacheMaxPage / 32
  uint32_t page_magic;     // 2^32 / page_blocks, rounded up
  int max_tokens;          // what the table holds of a sequence, 0 without pages
  int fmt;                 // 0 = E4M3, 1 = E5M2
};
constexpr int64_t kCacheMaxPage = 2048;

// rows of keys, values, queries or outputs: [T][heads][dim] at any distance of tokens and heads
struct CacheRows {
  const void* p;
  int64_t token, head;  // distances in elements
};

hipError_t mx_launch_cache_write(const CacheArgs& c, const CacheRows& k, const CacheRows& v,
                                 bool bf16, bool ceil, void* stream);
hipError_t mx_launch_cache_read(const CacheArgs& c, const CacheRows& k, const CacheRows& v,
                                bool bf16, void* stream);

constexpr int64_t kAttentionMaxRows = (int64_t)1 << 30;  // tokens x query heads
struct AttentionArgs {
  const void* q;
  void* out;
  float* lse;  // [T][heads] or NULL
  int64_t q_token, q_head, out_token, out_head;
  int heads, group;  // query heads, and how many share a head of the cache
  float scale_log2;
  bool bf16;
  void* stream;
  // set by the launcher
  int64_t slots;
  int4* where;
  float* part;
  float* stat;
};
// whether the kernels' 32-bit step numbers reach, if every sequence filled its table
bool mx_attention_fits(const CacheArgs& c, const AttentionArgs& a);
int64_t mx_attention_workspace_bytes(const CacheArgs& c, const AttentionArgs& a);
hipError_t mx_launch_cache_attention(const CacheArgs& c, AttentionArgs a, void* workspace);

// out[t] = base[t] + scaling[e] B[e] (A[e] x[t]), e = index[t]; a [E][r][K] and b [E][N][r] of x's type
constexpr int64_t kLoraMaxTokens = (int64_t)1 << 21, kLoraMaxRank = 128, kLoraMaxSize = (int64_t)1 << 26;
struct LoraArgs {
  const void* x;
  const void* a;
  const void* b;
  const int32_t* index;
  const float* scaling;  // [E] or NULL
  const void* base;      // or NULL
  void* out;
  float* h;              // workspace: [parts][T][r]
  int64_t ldx, ldb, ldo;
  int T, N, K, E, r;
  bool bf16, base_bf16, out_bf16, base_wide, out_wide;  // wide: rows at 16-byte addresses
  bool in_place;         // out is base
  void* stream;
  int parts, groups, slabs;  // set by the launcher, as small
  bool small;
};
// 0 where the call is one kernel
int64_t mx_lora_workspace_bytes(bool bf16, int64_t T, int64_t N, int64_t K, int64_t E, int64_t r);
hipError_t mx_launch_lora(LoraArgs a);
