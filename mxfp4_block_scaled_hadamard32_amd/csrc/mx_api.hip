// mx_api.hip — the extern "C" entry points declared in include/mx.h: argument validation and
// dispatch to the kernel launchers. No allocation, no synchronisation, no global state.
#include "mx.h"
#include "mx_launch.h"

namespace {

constexpr int32_t kVersion = 200;  // 0.2.0

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mx_status launch_status(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_LAUNCH; }

// scale row granularity of a GEMM operand: per row, per 32x32 tile or per 64x64 tile
bool granularity_ok(int32_t g) { return g == 1 || g == 32 || g == 64; }

mx_status check_opts(const mx_quant_opts* o) {
  if (!o) return MX_ERR_NULL;
  if (o->scale_rule != MX_SCALE_FLOOR && o->scale_rule != MX_SCALE_CEIL) return MX_ERR_ARG;
  if (o->round != MX_ROUND_RNE && o->round != MX_ROUND_SR) return MX_ERR_ARG;
  if (o->hadamard != 0 && o->hadamard != 1) return MX_ERR_ARG;
  return MX_OK;
}

// Source tensor checks shared by both quantizers: rows 16-byte aligned (8 elements per lane).
mx_status check_source(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
  if (dtype != MX_F32 && dtype != MX_BF16) return MX_ERR_ARG;
  if (rows < 0 || cols < 0 || ld < cols) return MX_ERR_SHAPE;
  const int64_t esize = dtype == MX_BF16 ? 2 : 4;
  if ((ld * esize) % 16 != 0) return MX_ERR_SHAPE;
  if (!aligned(x, 16)) return MX_ERR_ARG;
  return MX_OK;
}

mx_status gemm(const uint8_t* a, const uint8_t* as, int32_t ga, const uint8_t* b,
               const uint8_t* bs, int32_t gb, int64_t M, int64_t N, int64_t K, int32_t alpha_exp,
               int32_t out_dtype, void* c, int64_t ldc, void* stream) {
  if (M < 0 || N < 0 || K < 0) return MX_ERR_SHAPE;
  if (M % 32 || N % 32 || K % 32) return MX_ERR_SHAPE;
  if (ldc < N || ldc % 8 != 0) return MX_ERR_SHAPE;
  if (!granularity_ok(ga) || !granularity_ok(gb)) return MX_ERR_ARG;
  if (M % ga || N % gb) return MX_ERR_SHAPE;
  if (out_dtype != MX_F32 && out_dtype != MX_BF16) return MX_ERR_ARG;
  if (alpha_exp < -126 || alpha_exp > 127) return MX_ERR_ARG;
  if (M == 0 || N == 0) return MX_OK;
  if (!c) return MX_ERR_NULL;
  if (!aligned(c, 16)) return MX_ERR_ARG;
  if (K > 0) {
    if (!a || !as || !b || !bs) return MX_ERR_NULL;
    if (!aligned(a, 16) || !aligned(b, 16)) return MX_ERR_ARG;
  }
  GemmArgs g{a, as, ga, b, bs, gb, M, N, K, alpha_exp, out_dtype == MX_BF16, c, ldc, stream};
  return launch_status(mx_launch_gemm(g));
}

// rows of a norm operand: type-sized leading dimension and 16-byte rows
mx_status check_rows(const void* p, int64_t ld, int64_t cols, int32_t dtype) {
  const int64_t esize = dtype == MX_BF16 ? 2 : 4;
  if (ld < cols || (ld * esize) % 16 != 0) return MX_ERR_SHAPE;
  return aligned(p, 16) ? MX_OK : MX_ERR_ARG;
}

mx_status check_norm_sizes(int32_t dtype, int64_t rows, int64_t cols, int32_t gamma_dtype) {
  if (dtype != MX_F32 && dtype != MX_BF16) return MX_ERR_ARG;
  if (gamma_dtype != MX_F32 && gamma_dtype != MX_BF16) return MX_ERR_ARG;
  if (rows < 0 || cols < 0 || cols % 32 != 0) return MX_ERR_SHAPE;
  return cols > kNormMaxCols ? MX_ERR_UNSUPPORTED : MX_OK;
}

// `rows` rows of `width` bytes, `pitch` bytes apart
struct Rows {
  const void* p;
  int64_t pitch, width;
};

// Whether two operands have a byte in common. Rows that lie between one another (halves of one
// buffer) have none. A row of b starts v bytes after one of a; they meet when -b.width < v < a.width.
bool meet(const Rows& a, const Rows& b, int64_t rows) {
  if (!a.p || !b.p || rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  typedef __int128 wide;  // a caller's nonsense may pass 64 bits
  if (d >= (wide)(rows - 1) * a.pitch + a.width || -d >= (wide)(rows - 1) * b.pitch + b.width)
    return false;
  auto first = [&](int64_t from, int64_t least) {  // the least k >= least with from + k b.pitch > -b.width
    const int64_t x = -b.width - from;             // k > x / b.pitch
    const int64_t k = (x >= 0 ? x / b.pitch : -((-x + b.pitch - 1) / b.pitch)) + 1;
    return k > least ? k : least;
  };
  if (a.pitch == b.pitch) {  // only the difference of the rows' indexes matters
    const int64_t k = first(d, 1 - rows);
    return k < rows && d + k * b.pitch < a.width;
  }
  for (int64_t i = 0; i < rows; ++i) {
    const int64_t from = d - i * a.pitch, k = first(from, 0);
    if (k < rows && from + k * b.pitch < a.width) return true;
  }
  return false;
}

// whether `rows` rows have a byte in common with `size` bytes at p
bool meet_block(const Rows& a, const void* p, int64_t size, int64_t rows) {
  if (!a.p || !p || rows <= 0 || a.width <= 0 || size <= 0) return false;
  typedef __int128 wide;
  const wide d = (wide)reinterpret_cast<uintptr_t>(p) - (wide)reinterpret_cast<uintptr_t>(a.p);
  const wide i = d < a.width ? 0 : (d - a.width) / a.pitch + 1;  // the first row that ends behind p
  return i < rows && i * a.pitch < d + size;
}

// an output may be an input itself, or share nothing with it
bool clash(const Rows& out, const Rows& in, int64_t rows) {
  const bool same = out.p == in.p && (out.pitch == in.pitch || rows == 1);
  return !same && meet(out, in, rows);
}

// fmt 0: y only (required); 1, 2, 3: E2M1, E4M3, E5M2 codes, y optional
mx_status rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t dtype,
                  int64_t rows, int64_t cols, const void* gamma, int32_t gamma_dtype, float eps,
                  void* sum, int64_t lds, void* y, int64_t ldy, float* rstd, int fmt,
                  const mx_quant_opts* opts, uint8_t* codes, uint8_t* scales, void* stream) {
  mx_status s;
  if (fmt != 0 && (s = check_opts(opts)) != MX_OK) return s;
  if ((s = check_norm_sizes(dtype, rows, cols, gamma_dtype)) != MX_OK) return s;
  if (!(eps >= 0.0f) || eps > 3.402823466e+38f) return MX_ERR_ARG;
  if ((s = check_rows(x, ldx, cols, dtype)) != MX_OK) return s;
  if (residual && (s = check_rows(residual, ldr, cols, dtype)) != MX_OK) return s;
  if (sum && (s = check_rows(sum, lds, cols, dtype)) != MX_OK) return s;
  if ((y || fmt == 0) && (s = check_rows(y, ldy, cols, dtype)) != MX_OK) return s;
  if (!aligned(gamma, 16) || !aligned(rstd, 4) || !aligned(codes, fmt == 1 ? 16 : 8))
    return MX_ERR_ARG;
  if (rows == 0 || cols == 0) return MX_OK;
  if (!x || !gamma) return MX_ERR_NULL;
  if (fmt == 0 ? !y : (!codes || !scales)) return MX_ERR_NULL;
  const int64_t esize = dtype == MX_BF16 ? 2 : 4, width = cols * esize;
  const Rows rx{x, ldx * esize, width}, rr{residual, ldr * esize, width}, rs{sum, lds * esize, width},
      ry{y, ldy * esize, width};
  if (meet(rs, ry, rows) || clash(rs, rx, rows) || clash(rs, rr, rows) || clash(ry, rx, rows) ||
      clash(ry, rr, rows))
    return MX_ERR_ARG;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.gamma = gamma;
  a.sum = sum;
  a.y = y;
  a.rstd = rstd;
  a.codes = codes;
  a.scales = scales;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.ldr = ldr;
  a.lds = lds;
  a.ldy = ldy;
  a.eps = eps;
  a.fmt = fmt;
  a.bf16 = dtype == MX_BF16;
  a.gamma_bf16 = gamma_dtype == MX_BF16;
  if (fmt != 0) {
    a.seed = opts->seed;
    a.sign_mask = opts->sign_mask;
    a.ceil = opts->scale_rule == MX_SCALE_CEIL;
    a.sr = opts->round == MX_ROUND_SR;
    a.hadamard = opts->hadamard == 1;
  }
  a.stream = stream;
  return launch_status(mx_launch_rmsnorm(a));
}

// the cache of a call and its T rows, checked and as the kernels take it
mx_status cache_args(const mx_cache* c, int64_t T, CacheArgs& o) {
  if (!c) return MX_ERR_NULL;
  if (T < 0 || c->n_pages < 0 || c->seqs < 0 || c->table_width < 0 || c->heads < 0) return MX_ERR_SHAPE;
  if (c->fmt != MX_E4M3 && c->fmt != MX_E5M2) return MX_ERR_ARG;
  if (c->page_size <= 0 || c->page_size % 32 || c->page_size > kCacheMaxPage) return MX_ERR_ARG;
  if (c->dim != 64 && c->dim != 128 && c->dim != 192 && c->dim != 256) return MX_ERR_UNSUPPORTED;
  if (c->seqs > ((int64_t)1 << 20) || T > ((int64_t)1 << 24) || c->heads > 65535 ||
      c->n_pages > 0x7FFFFFFF || c->table_width > 0x7FFFFFFF)
    return MX_ERR_UNSUPPORTED;
  if (!c->offsets && T != c->seqs) return MX_ERR_SHAPE;
  if (!aligned(c->kq, 16) || !aligned(c->vq, 16) || !aligned(c->pages, 4) ||
      !aligned(c->lengths, 4) || !aligned(c->offsets, 4))
    return MX_ERR_ARG;
  if (T > 0 && c->seqs > 0 && c->heads > 0) {
    if (!c->lengths || (c->table_width > 0 && !c->pages)) return MX_ERR_NULL;
    if (c->n_pages > 0 && (!c->kq || !c->ks || !c->vq || !c->vs)) return MX_ERR_NULL;
  }
  o.kq = c->kq;
  o.ks = c->ks;
  o.vq = c->vq;
  o.vs = c->vs;
  o.pages = c->pages;
  o.lengths = c->lengths;
  o.offsets = c->offsets;
  o.n_pages = (int)c->n_pages;
  o.seqs = (int)c->seqs;
  o.table_width = (int)c->table_width;
  o.heads = c->heads;
  o.dim = c->dim;
  o.rows = (int)T;
  o.page_blocks = c->page_size / 32;
  o.page_magic = (uint32_t)((((uint64_t)1 << 32) + o.page_blocks - 1) / o.page_blocks);
  const int64_t tokens = c->table_width * c->page_size, most = 0x7FFFFF00;
  o.max_tokens = c->n_pages == 0 ? 0 : (int)(tokens < most ? tokens : most);
  o.fmt = c->fmt;
  return MX_OK;
}

// rows [T][heads][dim] and the bytes from the first to the last of them
mx_status cache_rows(const mx_rows* r, int32_t dtype, int64_t T, int64_t heads, int64_t dim,
                     CacheRows& o, Rows& span) {
  if (!r) return MX_ERR_NULL;
  if (dtype != MX_F32 && dtype != MX_BF16) return MX_ERR_ARG;
  const int64_t esize = dtype == MX_BF16 ? 2 : 4, most = (int64_t)1 << 40;
  if (!aligned(r->p, 16)) return MX_ERR_ARG;
  if (r->token > most || r->head > most) return MX_ERR_SHAPE;
  if (T > 0 && heads > 1 && (r->head < dim || (r->head * esize) % 16)) return MX_ERR_SHAPE;
  if (heads > 0 && T > 1 && (r->token < dim || (r->token * esize) % 16)) return MX_ERR_SHAPE;
  // one of the two distances holds all rows of the other: [T][heads] or [heads][T]
  if (T > 1 && heads > 1 && r->token < (heads - 1) * r->head + dim &&
      r->head < (T - 1) * r->token + dim)
    return MX_ERR_SHAPE;
  if (T > 0 && heads > 0 && !r->p) return MX_ERR_NULL;
  o = CacheRows{r->p, T > 1 ? r->token : 0, heads > 1 ? r->head : 0};
  span = T > 0 && heads > 0
             ? Rows{r->p, 1, ((T - 1) * o.token + (heads - 1) * o.head + dim) * esize}
             : Rows{nullptr, 1, 0};
  return MX_OK;
}

// the T rows of two operands share a byte: whole extents, but rows that lie between one another
// (token after token in one buffer, at the same distance) may
bool rows_meet(const CacheRows& a, const Rows& sa, int64_t ha, const CacheRows& b, const Rows& sb,
               int64_t hb, int64_t T, int64_t dim, int64_t esize) {
  const int64_t wa = ((ha - 1) * a.head + dim) * esize, wb = ((hb - 1) * b.head + dim) * esize;
  if (!sa.p || !sb.p) return false;
  if (T > 1 && wa <= a.token * esize && wb <= b.token * esize)
    return meet(Rows{a.p, a.token * esize, wa}, Rows{b.p, b.token * esize, wb}, T);
  return meet(sa, sb, 1);
}

// rows inside the cache
bool meets_cache(const Rows& span, const CacheArgs& c) {
  const int64_t blocks = (int64_t)c.n_pages * c.heads * c.page_blocks, bytes = blocks * 32 * c.dim;
  return meet(span, Rows{c.kq, 1, bytes}, 1) || meet(span, Rows{c.vq, 1, bytes}, 1) ||
         meet(span, Rows{c.ks, 1, blocks}, 1) || meet(span, Rows{c.vs, 1, blocks}, 1);
}

// `rows` rows on the tables of the cache
bool meets_tables(const Rows& r, int64_t rows, const CacheArgs& c) {
  return meet_block(r, c.pages, (int64_t)c.seqs * c.table_width * 4, rows) ||
         meet_block(r, c.lengths, (int64_t)c.seqs * 4, rows) ||
         meet_block(r, c.offsets, ((int64_t)c.seqs + 1) * 4, rows);
}
// the T tokens' rows of an output on the tables: token by token, or all that lies between them where
// tokens are closer than their heads
bool meets_tables(const CacheRows& o, const Rows& span, int64_t T, int64_t heads, int64_t esize,
                  const CacheArgs& c) {
  const int64_t width = ((heads - 1) * o.head + c.dim) * esize;
  return T > 1 && width <= o.token * esize ? meets_tables(Rows{o.p, o.token * esize, width}, T, c)
                                           : meets_tables(span, 1, c);
}

}  // namespace

extern "C" {

mx_status mx_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                      int32_t axis, const mx_quant_opts* opts, uint8_t* codes, uint8_t* scales,
                      void* stream) {
  mx_status s = check_opts(opts);
  if (s != MX_OK) return s;
  if (axis != 0 && axis != 1) return MX_ERR_ARG;
  if ((s = check_source(x, dtype, rows, cols, ld)) != MX_OK) return s;
  if (axis == 1 && cols % 32 != 0) return MX_ERR_SHAPE;
  if (axis == 0 && (rows % 32 != 0 || cols % 8 != 0)) return MX_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MX_OK;
  if (!x || !codes || !scales) return MX_ERR_NULL;
  // rows: the 16 code bytes of a block per lane; columns: 16-byte pieces of transposed code rows
  if (!aligned(codes, 16)) return MX_ERR_ARG;
  QuantArgs a{x, dtype == MX_BF16, rows, cols, ld, axis, opts->scale_rule == MX_SCALE_CEIL,
              opts->round == MX_ROUND_SR, opts->hadamard == 1, opts->sign_mask, opts->seed,
              codes, scales, nullptr, nullptr, stream};
  return launch_status(mx_launch_quantize(a));
}

mx_status mx_quantize_2d(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                         const mx_quant_opts* opts, uint8_t* codes, uint8_t* scales,
                         uint8_t* codes_t, uint8_t* scales_t, void* stream) {
  mx_status s = check_opts(opts);
  if (s != MX_OK) return s;
  if (opts->hadamard) return MX_ERR_UNSUPPORTED;
  if ((s = check_source(x, dtype, rows, cols, ld)) != MX_OK) return s;
  if (rows % 32 != 0 || cols % 32 != 0) return MX_ERR_SHAPE;
  if ((codes_t == nullptr) != (scales_t == nullptr)) return MX_ERR_NULL;
  if (rows == 0 || cols == 0) return MX_OK;
  if (!x || !codes || !scales) return MX_ERR_NULL;
  if (!aligned(codes, 16) || (codes_t && !aligned(codes_t, 16))) return MX_ERR_ARG;
  QuantArgs a{x, dtype == MX_BF16, rows, cols, ld, 1, opts->scale_rule == MX_SCALE_CEIL,
              opts->round == MX_ROUND_SR, false, 0u, opts->seed, codes, scales, codes_t,
              scales_t, stream};
  return launch_status(mx_launch_quantize_2d(a));
}

mx_status mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                        int32_t block_rows, int32_t inv_hadamard, uint32_t sign_mask, float* out,
                        void* stream) {
  if (rows < 0 || cols < 0 || cols % 32 != 0) return MX_ERR_SHAPE;
  if (block_rows != 1 && block_rows != 32) return MX_ERR_ARG;
  if (inv_hadamard != 0 && inv_hadamard != 1) return MX_ERR_ARG;
  if (inv_hadamard && block_rows != 1) return MX_ERR_UNSUPPORTED;
  if (block_rows == 32 && rows % 32 != 0) return MX_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MX_OK;
  if (!codes || !scales || !out) return MX_ERR_NULL;
  if (!aligned(codes, 4) || !aligned(out, 16)) return MX_ERR_ARG;
  return launch_status(mx_launch_dequantize(codes, scales, rows, cols, block_rows, inv_hadamard,
                                            sign_mask, out, stream));
}

mx_status mx_gemm_fprop_quant(const uint8_t* xq, const uint8_t* xs, int32_t gx, const uint8_t* wq,
                              const uint8_t* ws, int32_t gw, int64_t T, int64_t N, int64_t K,
                              int32_t alpha_exp, const mx_quant_opts* opts, uint8_t* yq,
                              uint8_t* ys, void* stream) {
  mx_status s = check_opts(opts);
  if (s != MX_OK) return s;
  if (T < 0 || N < 0 || K < 0) return MX_ERR_SHAPE;
  if (T % 32 || N % 32 || K % 32) return MX_ERR_SHAPE;
  if (!granularity_ok(gx) || !granularity_ok(gw)) return MX_ERR_ARG;
  if (T % gx || N % gw) return MX_ERR_SHAPE;
  if (alpha_exp < -126 || alpha_exp > 127) return MX_ERR_ARG;
  if (T == 0 || N == 0) return MX_OK;
  if (K == 0 || K % 128 != 0) return MX_ERR_UNSUPPORTED;  // the streaming kernels only
  if (!xq || !xs || !wq || !ws || !yq || !ys) return MX_ERR_NULL;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(yq, 4)) return MX_ERR_ARG;
  GemmArgs g{xq, xs, gx, wq, ws, gw, T, N, K, alpha_exp, false, nullptr, N, stream};
  GemmQuantOut q{yq, ys, opts->hadamard == 1, opts->round == MX_ROUND_SR,
                 opts->scale_rule == MX_SCALE_CEIL, opts->sign_mask, opts->seed};
  return launch_status(mx_launch_gemm_quant(g, q));
}

mx_status mx_gemm_fprop(const uint8_t* xq, const uint8_t* xs, int32_t gx, const uint8_t* wq,
                        const uint8_t* ws, int32_t gw, int64_t T, int64_t N, int64_t K,
                        int32_t alpha_exp, int32_t out_dtype, void* y, int64_t ldy, void* stream) {
  return gemm(xq, xs, gx, wq, ws, gw, T, N, K, alpha_exp, out_dtype, y, ldy, stream);
}

mx_status mx_gemm_dgrad(const uint8_t* dyq, const uint8_t* dys, int32_t gdy, const uint8_t* wtq,
                        const uint8_t* wts, int32_t gwt, int64_t T, int64_t K, int64_t N,
                        int32_t alpha_exp, int32_t out_dtype, void* dx, int64_t ldx, void* stream) {
  return gemm(dyq, dys, gdy, wtq, wts, gwt, T, K, N, alpha_exp, out_dtype, dx, ldx, stream);
}

mx_status mx_gemm_wgrad(const uint8_t* dytq, const uint8_t* dyts, int32_t gdy, const uint8_t* xtq,
                        const uint8_t* xts, int32_t gx, int64_t N, int64_t K, int64_t T,
                        int32_t alpha_exp, int32_t out_dtype, void* dw, int64_t ldw, void* stream) {
  return gemm(dytq, dyts, gdy, xtq, xts, gx, N, K, T, alpha_exp, out_dtype, dw, ldw, stream);
}

mx_status mx_quantize_mxfp8(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                            int32_t axis, int32_t fmt, const mx_quant_opts* opts, uint8_t* codes,
                            uint8_t* scales, void* stream) {
  mx_status s = check_opts(opts);
  if (s != MX_OK) return s;
  if (axis != 0 && axis != 1) return MX_ERR_ARG;
  if (fmt != MX_E4M3 && fmt != MX_E5M2) return MX_ERR_ARG;
  if ((s = check_source(x, dtype, rows, cols, ld)) != MX_OK) return s;
  if (axis == 1 && cols % 32 != 0) return MX_ERR_SHAPE;
  if (axis == 0 && (rows % 32 != 0 || cols % 8 != 0)) return MX_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MX_OK;
  if (!x || !codes || !scales) return MX_ERR_NULL;
  // rows: 8 code bytes per lane; columns: 16-byte pieces of transposed code rows
  if (!aligned(codes, axis == 1 ? 8 : 16)) return MX_ERR_ARG;
  QuantArgs a{x, dtype == MX_BF16, rows, cols, ld, axis, opts->scale_rule == MX_SCALE_CEIL,
              opts->round == MX_ROUND_SR, opts->hadamard == 1, opts->sign_mask, opts->seed,
              codes, scales, nullptr, nullptr, stream};
  return launch_status(mx_launch_quantize_fp8(a, fmt));
}

mx_status mx_gemm_mxfp8(const uint8_t* aq, const uint8_t* as, int32_t afmt, const uint8_t* bq,
                        const uint8_t* bs, int32_t bfmt, int64_t M, int64_t N, int64_t K,
                        int32_t alpha_exp, int32_t out_dtype, void* c, int64_t ldc, void* stream) {
  if (M < 0 || N < 0 || K < 0) return MX_ERR_SHAPE;
  if (M % 32 || N % 32 || K % 32) return MX_ERR_SHAPE;
  if (ldc < N || ldc % 8 != 0) return MX_ERR_SHAPE;
  if ((afmt != MX_E4M3 && afmt != MX_E5M2) || (bfmt != MX_E4M3 && bfmt != MX_E5M2)) return MX_ERR_ARG;
  if (out_dtype != MX_F32 && out_dtype != MX_BF16) return MX_ERR_ARG;
  if (alpha_exp < -126 || alpha_exp > 127) return MX_ERR_ARG;
  if (M == 0 || N == 0) return MX_OK;
  if (!c) return MX_ERR_NULL;
  if (!aligned(c, 16)) return MX_ERR_ARG;
  GemmArgs g{aq, as, 1, bq, bs, 1, M, N, K, alpha_exp, out_dtype == MX_BF16, c, ldc, stream};
  if (K == 0) return launch_status(mx_launch_gemm(g));  // an empty sum: the output is zero
  if (K % 128 != 0) return MX_ERR_UNSUPPORTED;
  if (!aq || !as || !bq || !bs) return MX_ERR_NULL;
  if (!aligned(aq, 16) || !aligned(bq, 16)) return MX_ERR_ARG;
  return launch_status(mx_launch_gemm_fp8(g, afmt, bfmt));
}

mx_status mx_quantize_2d_blocks(const void* x, int32_t dtype, int64_t rows, int64_t cols,
                                int64_t ld, int32_t block, const mx_quant_opts* opts,
                                uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                                uint8_t* scales_t, void* stream) {
  mx_status s = check_opts(opts);
  if (s != MX_OK) return s;
  if (block != 8 && block != 32 && block != 64) return MX_ERR_ARG;
  if (opts->hadamard) return MX_ERR_UNSUPPORTED;
  if ((s = check_source(x, dtype, rows, cols, ld)) != MX_OK) return s;
  const int64_t unit = block > 32 ? block : 32;
  if (rows % unit != 0 || cols % unit != 0) return MX_ERR_SHAPE;
  if ((codes_t == nullptr) != (scales_t == nullptr)) return MX_ERR_NULL;
  if (rows == 0 || cols == 0) return MX_OK;
  if (!x || !codes || !scales) return MX_ERR_NULL;
  if (!aligned(codes, 16) || (codes_t && !aligned(codes_t, 16))) return MX_ERR_ARG;
  if (!aligned(scales, 4) || (scales_t && !aligned(scales_t, 4))) return MX_ERR_ARG;
  QuantArgs a{x, dtype == MX_BF16, rows, cols, ld, 1, opts->scale_rule == MX_SCALE_CEIL,
              opts->round == MX_ROUND_SR, false, 0u, opts->seed, codes, scales, codes_t,
              scales_t, stream};
  return launch_status(mx_launch_quantize_2d_blocks(a, block));
}

mx_status mx_scale_mismatch_map(const void* x, int32_t dtype, int64_t rows, int64_t cols,
                                int64_t ld, int32_t scale_rule, int8_t* map, void* stream) {
  if (scale_rule != MX_SCALE_FLOOR && scale_rule != MX_SCALE_CEIL) return MX_ERR_ARG;
  mx_status s = check_source(x, dtype, rows, cols, ld);
  if (s != MX_OK) return s;
  if (rows % 32 != 0 || cols % 32 != 0) return MX_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MX_OK;
  if (!x || !map) return MX_ERR_NULL;
  if (!aligned(map, 8)) return MX_ERR_ARG;
  return launch_status(mx_launch_scale_mismatch(x, dtype == MX_BF16, rows, cols, ld,
                                                scale_rule == MX_SCALE_CEIL, map, stream));
}

mx_status mx_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t dtype,
                     int64_t rows, int64_t cols, const void* gamma, int32_t gamma_dtype, float eps,
                     void* sum, int64_t lds, void* y, int64_t ldy, float* rstd, void* stream) {
  return rmsnorm(x, ldx, residual, ldr, dtype, rows, cols, gamma, gamma_dtype, eps, sum, lds, y,
                 ldy, rstd, 0, nullptr, nullptr, nullptr, stream);
}

mx_status mx_rmsnorm_quant(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                           int32_t dtype, int64_t rows, int64_t cols, const void* gamma,
                           int32_t gamma_dtype, float eps, void* sum, int64_t lds, void* y,
                           int64_t ldy, float* rstd, const mx_quant_opts* opts, uint8_t* codes,
                           uint8_t* scales, void* stream) {
  return rmsnorm(x, ldx, residual, ldr, dtype, rows, cols, gamma, gamma_dtype, eps, sum, lds, y,
                 ldy, rstd, 1, opts, codes, scales, stream);
}

mx_status mx_rmsnorm_quant_mxfp8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                 int32_t dtype, int64_t rows, int64_t cols, const void* gamma,
                                 int32_t gamma_dtype, float eps, void* sum, int64_t lds, void* y,
                                 int64_t ldy, float* rstd, int32_t fmt, const mx_quant_opts* opts,
                                 uint8_t* codes, uint8_t* scales, void* stream) {
  if (fmt != MX_E4M3 && fmt != MX_E5M2) return MX_ERR_ARG;
  return rmsnorm(x, ldx, residual, ldr, dtype, rows, cols, gamma, gamma_dtype, eps, sum, lds, y,
                 ldy, rstd, 2 + fmt, opts, codes, scales, stream);
}

int64_t mx_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols % 32 != 0 || cols > kNormMaxCols) return 0;
  return mx_norm_backward_blocks(rows, cols) * cols * (int64_t)sizeof(float);
}

mx_status mx_rmsnorm_backward(const void* dy, int64_t lddy, const void* dsum, int64_t ldds,
                              const void* s, int64_t lds, int32_t dtype, int64_t rows,
                              int64_t cols, const void* gamma, int32_t gamma_dtype,
                              const float* rstd, void* dx, int64_t lddx, float* dgamma,
                              void* workspace, int64_t workspace_bytes, void* stream) {
  mx_status st = check_norm_sizes(dtype, rows, cols, gamma_dtype);
  if (st != MX_OK) return st;
  if ((st = check_rows(dy, lddy, cols, dtype)) != MX_OK) return st;
  if (dsum && (st = check_rows(dsum, ldds, cols, dtype)) != MX_OK) return st;
  if ((st = check_rows(s, lds, cols, dtype)) != MX_OK) return st;
  if ((st = check_rows(dx, lddx, cols, dtype)) != MX_OK) return st;
  if (!aligned(gamma, 16) || !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(workspace, 16))
    return MX_ERR_ARG;
  if (cols == 0 || (rows == 0 && !dgamma)) return MX_OK;
  if (rows > 0) {
    if (!dy || !s || !gamma || !rstd || !dx) return MX_ERR_NULL;
    const int64_t need = dgamma ? mx_rmsnorm_backward_workspace(rows, cols) : 0;
    if (need > 0 && !workspace) return MX_ERR_NULL;
    if (workspace_bytes < need) return MX_ERR_ARG;
    const int64_t esize = dtype == MX_BF16 ? 2 : 4, width = cols * esize;
    const Rows rdx{dx, lddx * esize, width}, rdy{dy, lddy * esize, width}, rs{s, lds * esize, width},
        rds{dsum, ldds * esize, width};
    // dgamma reads dy and s beside the rows that are written
    if (dgamma ? meet(rdx, rdy, rows) || meet(rdx, rs, rows)
               : clash(rdx, rdy, rows) || clash(rdx, rs, rows))
      return MX_ERR_ARG;
    if (clash(rdx, rds, rows)) return MX_ERR_ARG;
  }
  NormBackwardArgs a{dy,   dsum, s,    gamma, rstd, dx,   dgamma, dgamma ? (float*)workspace : nullptr,
                     rows, cols, lddy, ldds,  lds,  lddx, dtype == MX_BF16,
                     gamma_dtype == MX_BF16, stream, 0.0f, 0};
  return launch_status(mx_launch_rmsnorm_backward(a));
}

mx_status mx_gemv(const void* x, int32_t dtype, int64_t ldx, const uint8_t* wq, const uint8_t* ws,
                  int32_t gw, int64_t T, int64_t N, int64_t K, int32_t hadamard,
                  uint32_t sign_mask, int32_t alpha_exp, int32_t out_dtype, void* y, int64_t ldy,
                  void* workspace, int64_t workspace_bytes, void* stream) {
  mx_status s = check_source(x, dtype, T, K, ldx);
  if (s != MX_OK) return s;
  if (N < 0 || K % 32 || ldy < N) return MX_ERR_SHAPE;
  if (!granularity_ok(gw)) return MX_ERR_ARG;
  if (N % gw) return MX_ERR_SHAPE;
  if (hadamard != 0 && hadamard != 1) return MX_ERR_ARG;
  if (out_dtype != MX_F32 && out_dtype != MX_BF16) return MX_ERR_ARG;
  if (alpha_exp < -126 || alpha_exp > 127) return MX_ERR_ARG;
  if (!aligned(y, out_dtype == MX_BF16 ? 2 : 4) || !aligned(wq, 16)) return MX_ERR_ARG;
  if (T == 0 || N == 0) return MX_OK;
  if (T > kGemvMaxTokens || N > kGemvMaxRows) return MX_ERR_UNSUPPORTED;
  if (!y || (K > 0 && (!x || !wq || !ws))) return MX_ERR_NULL;
  const int64_t esize = dtype == MX_BF16 ? 2 : 4, osize = out_dtype == MX_BF16 ? 2 : 4;
  if (meet(Rows{x, ldx * esize, K * esize}, Rows{y, ldy * osize, N * osize}, T)) return MX_ERR_ARG;
  const int64_t need = mx_gemv_workspace(dtype, T, N, K, hadamard, out_dtype);
  if (workspace && need > 0 && (workspace_bytes < need || !aligned(workspace, 16)))
    return MX_ERR_ARG;
  GemvArgs a{x, wq, ws, y, T, N, K, ldx, ldy, gw, alpha_exp, sign_mask, dtype == MX_BF16,
             hadamard == 1, out_dtype == MX_BF16, stream,
             need > 0 ? static_cast<float*>(workspace) : nullptr};
  return launch_status(mx_launch_gemv(a));
}

int64_t mx_gemv_workspace(int32_t dtype, int64_t T, int64_t N, int64_t K, int32_t hadamard,
                          int32_t out_dtype) {
  if (T <= 0 || N <= 0 || K <= 0 || T > kGemvMaxTokens || N > kGemvMaxRows) return 0;
  return mx_gemv_workspace_bytes(T, N, K, dtype == MX_BF16, hadamard == 1, out_dtype == MX_BF16);
}

mx_status mx_cache_write(const mx_rows* k, const mx_rows* v, int32_t dtype, int64_t T,
                         const mx_cache* cache, int32_t scale_rule, void* stream) {
  if (scale_rule != MX_SCALE_FLOOR && scale_rule != MX_SCALE_CEIL) return MX_ERR_ARG;
  CacheArgs c{};
  CacheRows rk, rv;
  Rows sk, sv;
  mx_status s = cache_args(cache, T, c);
  if (s != MX_OK) return s;
  if ((s = cache_rows(k, dtype, T, c.heads, c.dim, rk, sk)) != MX_OK) return s;
  if ((s = cache_rows(v, dtype, T, c.heads, c.dim, rv, sv)) != MX_OK) return s;
  if (meets_cache(sk, c) || meets_cache(sv, c)) return MX_ERR_ARG;
  if (T == 0 || c.seqs == 0 || c.heads == 0 || c.max_tokens == 0) return MX_OK;
  return launch_status(mx_launch_cache_write(c, rk, rv, dtype == MX_BF16, scale_rule == MX_SCALE_CEIL,
                                             stream));
}

mx_status mx_cache_read(const mx_rows* k, const mx_rows* v, int32_t dtype, int64_t T,
                        const mx_cache* cache, void* stream) {
  CacheArgs c{};
  CacheRows rk, rv;
  Rows sk, sv;
  mx_status s = cache_args(cache, T, c);
  if (s != MX_OK) return s;
  if ((s = cache_rows(k, dtype, T, c.heads, c.dim, rk, sk)) != MX_OK) return s;
  if ((s = cache_rows(v, dtype, T, c.heads, c.dim, rv, sv)) != MX_OK) return s;
  const int64_t esize = dtype == MX_BF16 ? 2 : 4;
  if (meets_cache(sk, c) || meets_cache(sv, c) ||
      rows_meet(rk, sk, c.heads, rv, sv, c.heads, T, c.dim, esize))
    return MX_ERR_ARG;
  if (T == 0 || c.seqs == 0 || c.heads == 0) return MX_OK;
  if (meets_tables(rk, sk, T, c.heads, esize, c) || meets_tables(rv, sv, T, c.heads, esize, c))
    return MX_ERR_ARG;
  return launch_status(mx_launch_cache_read(c, rk, rv, dtype == MX_BF16, stream));
}

int64_t mx_cache_attention_workspace(int64_t T, int64_t q_heads, const mx_cache* cache) {
  CacheArgs c{};
  if (cache_args(cache, T, c) != MX_OK || q_heads < 0 || q_heads > 65535 ||
      T * q_heads > kAttentionMaxRows)
    return -1;
  if (T == 0 || q_heads == 0 || c.seqs == 0) return 0;
  if (c.heads == 0 || q_heads % c.heads) return -1;
  AttentionArgs a{};
  a.heads = (int)q_heads;
  a.group = (int)q_heads / c.heads;
  return mx_attention_fits(c, a) ? mx_attention_workspace_bytes(c, a) : -1;
}

mx_status mx_cache_attention(const mx_rows* q, const mx_rows* out, float* lse, int32_t dtype,
                             int64_t T, int64_t q_heads, float scale, const mx_cache* cache,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  CacheArgs c{};
  CacheRows rq, ro;
  Rows sq, so;
  mx_status s = cache_args(cache, T, c);
  if (s != MX_OK) return s;
  if (q_heads < 0) return MX_ERR_SHAPE;
  if (q_heads > 65535) return MX_ERR_UNSUPPORTED;
  if (c.heads == 0 ? q_heads != 0 : q_heads % c.heads != 0) return MX_ERR_SHAPE;
  if (T * q_heads > kAttentionMaxRows) return MX_ERR_UNSUPPORTED;
  if (!(scale >= -3.402823466e+38f && scale <= 3.402823466e+38f)) return MX_ERR_ARG;
  if ((s = cache_rows(q, dtype, T, q_heads, c.dim, rq, sq)) != MX_OK) return s;
  if ((s = cache_rows(out, dtype, T, q_heads, c.dim, ro, so)) != MX_OK) return s;
  if (!aligned(lse, 4) || !aligned(workspace, 16)) return MX_ERR_ARG;
  if (T == 0 || q_heads == 0 || c.seqs == 0) return MX_OK;
  const int64_t esize = dtype == MX_BF16 ? 2 : 4;
  const Rows sl{lse, 1, T * q_heads * 4};
  if (rows_meet(rq, sq, q_heads, ro, so, q_heads, T, c.dim, esize) || meets_cache(so, c) ||
      meets_cache(sl, c) || meet(sl, so, 1) || meet(sl, sq, 1) ||
      meets_tables(ro, so, T, q_heads, esize, c) || meets_tables(sl, 1, c))
    return MX_ERR_ARG;
  AttentionArgs a{rq.p, const_cast<void*>(ro.p), lse, rq.token, rq.head, ro.token, ro.head,
                  (int)q_heads, (int)q_heads / c.heads, scale * 1.4426950408889634f,
                  dtype == MX_BF16, stream, 0, nullptr, nullptr, nullptr};
  if (!mx_attention_fits(c, a)) return MX_ERR_UNSUPPORTED;
  const int64_t need = mx_attention_workspace_bytes(c, a);
  if (need > 0 && !workspace) return MX_ERR_NULL;
  if (workspace_bytes < need) return MX_ERR_ARG;
  return launch_status(mx_launch_cache_attention(c, a, workspace));
}

int64_t mx_lora_workspace(int32_t dtype, int64_t T, int64_t N, int64_t K, int64_t adapters,
                          int64_t rank) {
  if (T <= 0 || N <= 0 || N > kLoraMaxSize || K <= 0 || adapters <= 0 || rank <= 0 || T > kLoraMaxTokens || K > kLoraMaxSize ||
      adapters > kLoraMaxSize || rank > kLoraMaxRank)
    return 0;
  return mx_lora_workspace_bytes(dtype == MX_BF16, T, N, K, adapters, rank);
}

mx_status mx_lora(const void* x, int32_t dtype, int64_t ldx, const void* a, const void* b,
                  int64_t adapters, int64_t rank, const int32_t* index, const float* scaling,
                  const void* base, int32_t base_dtype, int64_t ldb, int64_t T, int64_t N, int64_t K,
                  int32_t out_dtype, void* out, int64_t ldo, void* workspace,
                  int64_t workspace_bytes, void* stream) {
  mx_status s = check_source(x, dtype, T, K, ldx);
  if (s != MX_OK) return s;
  if (N < 0 || adapters < 0 || rank < 0 || K % 8 || rank % 8 || ldo < N) return MX_ERR_SHAPE;
  if (out_dtype != MX_F32 && out_dtype != MX_BF16) return MX_ERR_ARG;
  if (base) {
    if (base_dtype != MX_F32 && base_dtype != MX_BF16) return MX_ERR_ARG;
    if (ldb < N) return MX_ERR_SHAPE;
    if (!aligned(base, base_dtype == MX_BF16 ? 2 : 4)) return MX_ERR_ARG;
  }
  if (!aligned(out, out_dtype == MX_BF16 ? 2 : 4) || !aligned(a, 16) || !aligned(b, 16) ||
      !aligned(index, 4) || !aligned(scaling, 4))
    return MX_ERR_ARG;
  if (rank > kLoraMaxRank || T > kLoraMaxTokens || N > kLoraMaxSize || K > kLoraMaxSize ||
      adapters > kLoraMaxSize)
    return MX_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return MX_OK;
  const bool any = adapters > 0 && rank > 0 && K > 0;  // else every adapter adds nothing
  if (!out || (any && (!x || !a || !b || !index))) return MX_ERR_NULL;
  const int64_t esize = dtype == MX_BF16 ? 2 : 4, osize = out_dtype == MX_BF16 ? 2 : 4,
                bsize = base_dtype == MX_BF16 ? 2 : 4;
  const Rows rx{x, ldx * esize, K * esize}, ro{out, ldo * osize, N * osize}, rb{base, ldb * bsize, N * bsize};
  const bool in_place = base == out && base_dtype == out_dtype && (ldb == ldo || T == 1);
  if (meet(rx, ro, T) || (!in_place && meet(rb, ro, T))) return MX_ERR_ARG;
  if (any && (meet_block(ro, a, adapters * rank * K * esize, T) ||
              meet_block(ro, b, adapters * rank * N * esize, T) || meet_block(ro, index, T * 4, T) ||
              meet_block(ro, scaling, adapters * 4, T)))
    return MX_ERR_ARG;
  const int64_t need = any ? mx_lora_workspace(dtype, T, N, K, adapters, rank) : 0;
  if (need > 0 && !workspace) return MX_ERR_NULL;
  if (need > 0 && (workspace_bytes < need || !aligned(workspace, 16))) return MX_ERR_ARG;
  auto wide = [](const void* p, int64_t ld, int64_t size) { return aligned(p, 16) && ld * size % 16 == 0; };
  LoraArgs l{x, a, b, index, scaling, base, out, static_cast<float*>(workspace), ldx, ldb, ldo,
             (int)T, (int)N, any ? (int)K : 0, any ? (int)adapters : 0, any ? (int)rank : 8,
             dtype == MX_BF16, base_dtype == MX_BF16, out_dtype == MX_BF16, wide(base, ldb, bsize),
             wide(out, ldo, osize), in_place, stream, 0, 0, 0, false};
  return launch_status(mx_launch_lora(l));
}

const char* mx_status_string(int32_t status) {
  switch (status) {
    case MX_OK: return "MX_OK";
    case MX_ERR_NULL: return "MX_ERR_NULL: a required pointer is NULL";
    case MX_ERR_SHAPE: return "MX_ERR_SHAPE: bad dimension, multiple-of-32 rule or leading dimension";
    case MX_ERR_UNSUPPORTED: return "MX_ERR_UNSUPPORTED: option combination not defined";
    case MX_ERR_LAUNCH: return "MX_ERR_LAUNCH: the HIP runtime refused the launch";
    case MX_ERR_ARG: return "MX_ERR_ARG: option value out of range or misaligned pointer";
    default: return "unknown mx_status";
  }
}

int32_t mx_version(void) { return kVersion; }

}  // extern "C"
