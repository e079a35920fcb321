// Host layer of the packed forms and the RMS norm: argument checks (pure host functions, no HIP
// call), kernel choice, launch.
#include <cmath>

#include "host_check.h"
#include "packed.h"

using gdr::host::fail;
using gdr::host::log_enabled;
using gdr::host::ok;
using gdr::host::overlap;
using gdr::host::Range;
using gdr::host::rng;

namespace {

constexpr long long kMaxStreams = 1LL << 18;   // (sequence, value head) pairs: 2^31 work-items at Dv = 512
constexpr long long kMaxRows = 1LL << 26;      // (token, value head) pairs
constexpr long long kMaxStride = 1LL << 23;    // elements between the tokens of a packed tensor
constexpr int kMaxD = 16384;                   // channels of a norm's row

bool io_known(int t) { return t == GDR_F32 || t == GDR_BF16 || t == GDR_F16; }
long long io_bytes(int t) { return t == GDR_F32 ? 4 : 2; }
bool misaligned(const void *p, long long bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// bytes from the first element to behind the last of `rows` rows of `width` elements
long double span(long long rows, long long stride, long long width, long long e) {
  return rows <= 0 ? 0.0L : (static_cast<long double>(rows - 1) * stride + width) * e;
}

// the descriptor on its own
gdr_status_t check_packed_desc(const gdr_packed_desc_t *d) {
  if (d == nullptr) return fail(GDR_EINVAL, "desc must be non-NULL");
  if (d->struct_size != sizeof(gdr_packed_desc_t))
    return fail(GDR_EINVAL, "desc->struct_size = %u, expected %zu (ABI mismatch)", d->struct_size,
                sizeof(gdr_packed_desc_t));
  if (d->n_tokens < 0 || d->n_seqs < 0) return fail(GDR_EINVAL, "n_tokens = %d, n_seqs = %d", d->n_tokens, d->n_seqs);
  if (d->Hk < 1 || d->Hv < 1) return fail(GDR_EINVAL, "Hk = %d and Hv = %d must be >= 1", d->Hk, d->Hv);
  if (d->Hv % d->Hk != 0) return fail(GDR_EINVAL, "Hv = %d is no multiple of Hk = %d", d->Hv, d->Hk);
  if (d->Dk < 1 || d->Dv < 1) return fail(GDR_EINVAL, "Dk = %d and Dv = %d must be >= 1", d->Dk, d->Dv);
  if (d->Dk > 128 || d->Dv > 512) return fail(GDR_ENOTSUP, "Dk = %d (max 128), Dv = %d (max 512)", d->Dk, d->Dv);
  if (d->n_seqs > 65535 || d->Hv > 65535) return fail(GDR_ENOTSUP, "n_seqs = %d, Hv = %d (max 65535 each)", d->n_seqs, d->Hv);
  if (static_cast<long long>(d->n_seqs) * d->Hv > kMaxStreams)
    return fail(GDR_ENOTSUP, "n_seqs * Hv = %lld (max %lld)", static_cast<long long>(d->n_seqs) * d->Hv, kMaxStreams);
  if (static_cast<long long>(d->n_tokens) * d->Hv > kMaxRows)
    return fail(GDR_ENOTSUP, "n_tokens * Hv = %lld (max %lld)", static_cast<long long>(d->n_tokens) * d->Hv, kMaxRows);
  if (d->n_slots < 0) return fail(GDR_EINVAL, "n_slots = %d", d->n_slots);
  if (!io_known(d->io_dtype)) return fail(GDR_EINVAL, "io_dtype = %d", d->io_dtype);
  if (d->decay != GDR_DECAY_NONE && d->decay != GDR_DECAY_SCALAR)
    return fail(d->decay == GDR_DECAY_CHANNEL ? GDR_ENOTSUP : GDR_EINVAL, "decay = %d (NONE or SCALAR)", d->decay);
  if (d->qk_norm != 0 && d->qk_norm != 1) return fail(GDR_EINVAL, "qk_norm = %d", d->qk_norm);
  if (d->impl != GDR_IMPL_AUTO && d->impl != GDR_IMPL_GENERIC && d->impl != GDR_IMPL_MFMA)
    return fail(GDR_EINVAL, "impl = %d", d->impl);
  if (!std::isfinite(d->scale)) return fail(GDR_EINVAL, "scale must be finite");
  if (!(d->qk_eps >= 0.f) || !std::isfinite(d->qk_eps) || !(d->norm_eps >= 0.f) || !std::isfinite(d->norm_eps))
    return fail(GDR_EINVAL, "qk_eps and norm_eps must be finite and >= 0");
  const long long kw = static_cast<long long>(d->Hk) * d->Dk, vw = static_cast<long long>(d->Hv) * d->Dv;
  const struct { const char *name; int64_t stride; long long width; } strides[] = {
      {"q_stride", d->q_stride, kw}, {"k_stride", d->k_stride, kw}, {"v_stride", d->v_stride, vw},
      {"out_stride", d->out_stride, vw}, {"gate_stride", d->gate_stride, vw}};
  for (const auto &s : strides) {
    if (s.stride != 0 && s.stride < s.width)
      return fail(GDR_EINVAL, "%s = %lld is less than a row's %lld", s.name, static_cast<long long>(s.stride), s.width);
    // 64 rows within 32-bit byte offsets
    if (s.stride > kMaxStride || s.width > kMaxStride)
      return fail(GDR_ENOTSUP, "%s = %lld, a row's length %lld (max %lld)", s.name, static_cast<long long>(s.stride), s.width, kMaxStride);
  }
  return ok();
}

long long or_width(int64_t stride, long long width) { return stride != 0 ? stride : width; }

gdr::PackedArgs packed_args(const gdr_packed_desc_t *d, const gdr_packed_inputs_t *in, float *pool, void *out) {
  gdr::PackedArgs a{};
  const long long kw = static_cast<long long>(d->Hk) * d->Dk, vw = static_cast<long long>(d->Hv) * d->Dv;
  a.q = in->q; a.k = in->k; a.v = in->v;
  a.beta = in->beta;
  a.log_alpha = d->decay == GDR_DECAY_SCALAR ? in->log_alpha : nullptr;
  a.cu = in->cu_seqlens; a.index = in->state_index; a.has = in->has_state;
  a.norm_w = in->norm_weight; a.norm_z = in->norm_gate;
  a.pool = pool; a.out = out;
  a.qs = or_width(d->q_stride, kw); a.ks = or_width(d->k_stride, kw); a.vs = or_width(d->v_stride, vw);
  a.os = or_width(d->out_stride, vw); a.zs = or_width(d->gate_stride, vw);
  a.N = d->n_tokens; a.n_seqs = d->n_seqs; a.Hk = d->Hk; a.Hv = d->Hv; a.Dk = d->Dk; a.Dv = d->Dv;
  a.n_slots = d->n_slots; a.qk_norm = d->qk_norm;
  a.scale = d->scale; a.qk_eps = d->qk_eps; a.norm_eps = d->norm_eps;
  return a;
}

gdr_status_t check_norm_desc(const gdr_norm_desc_t *d, bool bwd) {
  if (d == nullptr) return fail(GDR_EINVAL, "desc must be non-NULL");
  if (d->struct_size != sizeof(gdr_norm_desc_t))
    return fail(GDR_EINVAL, "desc->struct_size = %u, expected %zu (ABI mismatch)", d->struct_size, sizeof(gdr_norm_desc_t));
  if (d->rows < 0 || d->D < 1) return fail(GDR_EINVAL, "rows = %d, D = %d", d->rows, d->D);
  if (d->D > kMaxD) return fail(GDR_ENOTSUP, "D = %d (max %d)", d->D, kMaxD);
  // a grid's work-items stay below 2^32, by the most lanes that a row of so many loads may take
  const int loads = (d->D + 16 / static_cast<int>(io_bytes(d->io_dtype)) - 1) / (16 / static_cast<int>(io_bytes(d->io_dtype)));
  const long long lanes = loads <= 16 ? 16 : loads <= 32 ? 32 : loads <= 128 ? 64 : loads <= 512 ? 256 : loads <= 1024 ? 512 : 1024;
  if (d->rows > (0xfffff000LL / lanes)) return fail(GDR_ENOTSUP, "rows = %d at D = %d (max %lld)", d->rows, d->D, 0xfffff000LL / lanes);
  if (!io_known(d->io_dtype)) return fail(GDR_EINVAL, "io_dtype = %d", d->io_dtype);
  if (d->out_kind != GDR_OUT_IO && d->out_kind != GDR_OUT_INT8 && d->out_kind != GDR_OUT_FP8)
    return fail(GDR_EINVAL, "out_kind = %d", d->out_kind);
  if (bwd && d->out_kind != GDR_OUT_IO) return fail(GDR_ENOTSUP, "the gradient of an 8-bit output");
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return fail(GDR_EINVAL, "eps must be finite and >= 0");
  const struct { const char *name; int64_t stride; } strides[] = {
      {"x_stride", d->x_stride}, {"residual_stride", d->residual_stride}, {"gate_stride", d->gate_stride}, {"dy_stride", d->dy_stride}};
  for (const auto &s : strides) {
    if (s.stride != 0 && s.stride < d->D)
      return fail(GDR_EINVAL, "%s = %lld is less than D = %d", s.name, static_cast<long long>(s.stride), d->D);
    if (s.stride > (1LL << 40)) return fail(GDR_ENOTSUP, "%s = %lld", s.name, static_cast<long long>(s.stride));
  }
  return ok();
}

uint64_t bwd_ws_bytes(const gdr_norm_desc_t &d) {
  return static_cast<uint64_t>(gdr::rms_norm_bwd_groups(d.rows, d.D, d.io_dtype)) * d.D * 4u;
}

// none of the written ranges may meet an input or another written one
gdr_status_t check_disjoint(const Range *written, int nw, const Range *inputs, int ni) {
  for (int i = 0; i < nw; ++i) {
    for (int j = 0; j < ni; ++j)
      if (overlap(written[i], inputs[j])) return fail(GDR_EINVAL, "%s overlaps %s", written[i].name, inputs[j].name);
    for (int j = i + 1; j < nw; ++j)
      if (overlap(written[i], written[j])) return fail(GDR_EINVAL, "%s overlaps %s", written[i].name, written[j].name);
  }
  return ok();
}

}  // namespace

extern "C" {

gdr_status_t gdr_validate_packed(const gdr_packed_desc_t *d, const gdr_packed_inputs_t *in, const float *pool,
                                 const void *out, const void *ws, uint64_t ws_bytes, int for_step) {
  gdr_status_t st = check_packed_desc(d);
  if (st != GDR_OK) return st;
  if (in == nullptr) return fail(GDR_EINVAL, "inputs must be non-NULL");
  const bool need = d->n_tokens > 0 && d->n_seqs > 0;
  if (need && (in->q == nullptr || in->k == nullptr || in->v == nullptr || in->beta == nullptr))
    return fail(GDR_EINVAL, "q, k, v and beta are required");
  if (need && out == nullptr) return fail(GDR_EINVAL, "out is required");
  if (d->decay == GDR_DECAY_SCALAR ? (need && in->log_alpha == nullptr) : in->log_alpha != nullptr)
    return fail(GDR_EINVAL, "log_alpha is given iff decay is SCALAR");
  if (in->cu_seqlens == nullptr && d->n_seqs > 0) {
    if (!for_step) return fail(GDR_EINVAL, "cu_seqlens is required");
    if (d->n_tokens != d->n_seqs)
      return fail(GDR_EINVAL, "without cu_seqlens every sequence is one token: n_tokens = %d, n_seqs = %d", d->n_tokens, d->n_seqs);
  }
  if (pool == nullptr) {
    if (for_step && d->n_seqs > 0) return fail(GDR_EINVAL, "the pool is required");
    if (d->n_slots != 0) return fail(GDR_EINVAL, "n_slots = %d without a pool", d->n_slots);
    if (in->has_state != nullptr) return fail(GDR_EINVAL, "has_state without a pool");
  } else if (in->state_index == nullptr && d->n_slots < d->n_seqs) {
    return fail(GDR_EINVAL, "without state_index sequence s uses slot s: n_slots = %d, n_seqs = %d", d->n_slots, d->n_seqs);
  }
  if (in->norm_gate != nullptr && in->norm_weight == nullptr) return fail(GDR_EINVAL, "norm_gate needs norm_weight");
  const long long e = io_bytes(d->io_dtype);
  const void *io_ptrs[] = {in->q, in->k, in->v, in->norm_weight, in->norm_gate, out};
  for (const void *p : io_ptrs)
    if (misaligned(p, e)) return fail(GDR_EINVAL, "misaligned io pointer");
  const void *w_ptrs[] = {in->beta, in->log_alpha, in->cu_seqlens, in->state_index, pool};
  for (const void *p : w_ptrs)
    if (misaligned(p, 4)) return fail(GDR_EINVAL, "misaligned 4-byte pointer");

  const long long N = d->n_tokens, kw = static_cast<long long>(d->Hk) * d->Dk, vw = static_cast<long long>(d->Hv) * d->Dv;
  const Range inputs[] = {
      rng("q", in->q, span(N, or_width(d->q_stride, kw), kw, e)), rng("k", in->k, span(N, or_width(d->k_stride, kw), kw, e)),
      rng("v", in->v, span(N, or_width(d->v_stride, vw), vw, e)), rng("beta", in->beta, 4.0L * N * d->Hv),
      rng("log_alpha", in->log_alpha, 4.0L * N * d->Hv), rng("cu_seqlens", in->cu_seqlens, 4.0L * (d->n_seqs + 1)),
      rng("state_index", in->state_index, 4.0L * d->n_seqs), rng("has_state", in->has_state, d->n_seqs),
      rng("norm_weight", in->norm_weight, static_cast<long double>(d->Dv) * e),
      rng("norm_gate", in->norm_gate, span(N, or_width(d->gate_stride, vw), vw, e))};
  const uint64_t need_ws = for_step ? 0 : gdr_packed_fwd_workspace_size(d);
  const Range written[] = {rng("out", out, span(N, or_width(d->out_stride, vw), vw, e)),
                           rng("pool", pool, 4.0L * d->n_slots * d->Hv * d->Dv * d->Dk),
                           rng("workspace", need_ws > 0 ? ws : nullptr, static_cast<long double>(need_ws))};
  if (need_ws > 0) {
    if (ws == nullptr) return fail(GDR_EINVAL, "workspace is required");
    if (ws_bytes < need_ws)
      return fail(GDR_EINVAL, "workspace_bytes = %llu, need %llu", static_cast<unsigned long long>(ws_bytes),
                  static_cast<unsigned long long>(need_ws));
    if (misaligned(ws, 256)) return fail(GDR_EINVAL, "workspace must be 256-byte aligned");
  }
  return check_disjoint(written, 3, inputs, 10);
}

int gdr_packed_fwd_impl(const gdr_packed_desc_t *d) {
  if (check_packed_desc(d) != GDR_OK) return -1;
  const bool chunked = gdr::packed_chunk_supports(*d);
  if (d->impl == GDR_IMPL_MFMA) return chunked ? GDR_IMPL_MFMA : -1;
  return chunked && d->impl != GDR_IMPL_GENERIC ? GDR_IMPL_MFMA : GDR_IMPL_GENERIC;
}

uint64_t gdr_packed_fwd_workspace_size(const gdr_packed_desc_t *d) {
  return gdr_packed_fwd_impl(d) == GDR_IMPL_MFMA ? gdr::packed_chunk_ws_bytes(*d) : 0;
}

gdr_status_t gdr_packed_fwd(const gdr_packed_desc_t *d, const gdr_packed_inputs_t *in, float *pool, void *out,
                            void *ws, uint64_t ws_bytes, void *stream) {
  const gdr_status_t st = gdr_validate_packed(d, in, pool, out, ws, ws_bytes, 0);
  if (st != GDR_OK) return st;
  const int impl = gdr_packed_fwd_impl(d);
  if (impl < 0)
    return fail(GDR_ENOTSUP, "the chunked kernel does not cover this descriptor (Dk = %d, Dv = %d)", d->Dk, d->Dv);
  if (d->n_seqs == 0) return ok();
  gdr::PackedArgs a = packed_args(d, in, pool, out);
  a.ws = static_cast<uint8_t *>(ws);
  if (log_enabled())
    std::fprintf(stderr, "[gdr] packed_fwd %s N=%d seqs=%d Hk=%d Hv=%d Dk=%d Dv=%d io=%d\n",
                 impl == GDR_IMPL_MFMA ? "mfma" : "generic", d->n_tokens, d->n_seqs, d->Hk, d->Hv, d->Dk, d->Dv, d->io_dtype);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  if (impl == GDR_IMPL_MFMA) {
    e = gdr::launch_packed_chunk(a, d->io_dtype, s);
    if (e == hipSuccess && a.norm_w != nullptr) e = gdr::launch_packed_norm(a, d->io_dtype, s);
  } else {
    e = gdr::launch_packed_recur(a, d->io_dtype, s);
  }
  if (e != hipSuccess) return fail(GDR_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

gdr_status_t gdr_packed_step(const gdr_packed_desc_t *d, const gdr_packed_inputs_t *in, float *pool, void *out,
                             void *stream) {
  const gdr_status_t st = gdr_validate_packed(d, in, pool, out, nullptr, 0, 1);
  if (st != GDR_OK) return st;
  if (d->n_seqs == 0) return ok();
  if (log_enabled())
    std::fprintf(stderr, "[gdr] packed_step N=%d seqs=%d Hk=%d Hv=%d Dk=%d Dv=%d io=%d\n", d->n_tokens, d->n_seqs, d->Hk,
                 d->Hv, d->Dk, d->Dv, d->io_dtype);
  const hipError_t e = gdr::launch_packed_recur(packed_args(d, in, pool, out), d->io_dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(GDR_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

gdr_status_t gdr_validate_norm(const gdr_norm_desc_t *d, const void *x, const void *res, const void *w, const void *z,
                               const void *y, const float *scales, const void *res_out) {
  gdr_status_t st = check_norm_desc(d, false);
  if (st != GDR_OK) return st;
  const bool need = d->rows > 0, codes = d->out_kind != GDR_OUT_IO;
  if (need && (x == nullptr || y == nullptr)) return fail(GDR_EINVAL, "x and y are required");
  if (codes ? (need && scales == nullptr) : scales != nullptr)
    return fail(GDR_EINVAL, "scales are given iff the output has 8 bits");
  if ((res == nullptr) != (res_out == nullptr)) return fail(GDR_EINVAL, "residual and residual_out are given together");
  const long long e = io_bytes(d->io_dtype);
  const void *io_ptrs[] = {x, res, w, z, res_out, codes ? nullptr : y};
  for (const void *p : io_ptrs)
    if (misaligned(p, e)) return fail(GDR_EINVAL, "misaligned io pointer");
  if (misaligned(scales, 4)) return fail(GDR_EINVAL, "scales misaligned");
  const long long xs = or_width(d->x_stride, d->D), rs = or_width(d->residual_stride, d->D);
  const long double flat = static_cast<long double>(d->rows) * d->D;
  const Range r_x = rng("x", x, span(d->rows, xs, d->D, e)), r_res = rng("residual", res, span(d->rows, rs, d->D, e));
  // in place, row by row: the sum over x or residual, a plain output over x
  const bool same_rows = xs == d->D;
  const bool y_on_x = y == x && !codes && same_rows && res == nullptr;
  const bool sum_on_x = res != nullptr && res_out == x && same_rows, sum_on_res = res != nullptr && res_out == res && rs == d->D;
  const Range r_y = rng("y", y, flat * (codes ? 1 : e)), r_sum = rng("residual_out", res_out, flat * e),
              r_sc = rng("scales", scales, 4.0L * d->rows);
  const Range r_w = rng("weight", w, static_cast<long double>(d->D) * e), r_z = rng("gate", z, span(d->rows, or_width(d->gate_stride, d->D), d->D, e));
  if (overlap(r_y, r_x) && !y_on_x) return fail(GDR_EINVAL, "y overlaps x");
  if (overlap(r_y, r_res)) return fail(GDR_EINVAL, "y overlaps residual");
  if (overlap(r_sum, r_x) && !sum_on_x) return fail(GDR_EINVAL, "residual_out overlaps x");
  if (overlap(r_sum, r_res) && !sum_on_res) return fail(GDR_EINVAL, "residual_out overlaps residual");
  const Range written[] = {r_y, r_sum, r_sc}, others[] = {r_w, r_z};
  st = check_disjoint(written, 3, others, 2);
  if (st != GDR_OK) return st;
  if (overlap(r_sc, r_x) || overlap(r_sc, r_res)) return fail(GDR_EINVAL, "scales overlap an input");
  return ok();
}

gdr_status_t gdr_rms_norm(const gdr_norm_desc_t *d, const void *x, const void *res, const void *w, const void *z,
                          void *y, float *scales, void *res_out, void *stream) {
  const gdr_status_t st = gdr_validate_norm(d, x, res, w, z, y, scales, res_out);
  if (st != GDR_OK) return st;
  gdr::NormArgs a{};
  a.x = x; a.res = res; a.w = w; a.z = z; a.y = y; a.scales = scales; a.res_out = res_out;
  a.xs = or_width(d->x_stride, d->D); a.rs = or_width(d->residual_stride, d->D); a.zs = or_width(d->gate_stride, d->D);
  a.rows = d->rows; a.D = d->D; a.out_kind = d->out_kind; a.eps = d->eps; a.inv_d = 1.f / d->D;
  if (log_enabled())
    std::fprintf(stderr, "[gdr] rms_norm rows=%d D=%d io=%d out=%d\n", d->rows, d->D, d->io_dtype, d->out_kind);
  const hipError_t e = gdr::launch_rms_norm(a, d->io_dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(GDR_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

uint64_t gdr_rms_norm_bwd_workspace_size(const gdr_norm_desc_t *d) {
  return check_norm_desc(d, true) == GDR_OK ? bwd_ws_bytes(*d) : 0;
}

gdr_status_t gdr_validate_norm_bwd(const gdr_norm_desc_t *d, const void *x, const void *dy, const void *w, const void *z,
                                   const void *d_res, const void *dx, const float *dw, const void *dz, const void *ws,
                                   uint64_t ws_bytes) {
  gdr_status_t st = check_norm_desc(d, true);
  if (st != GDR_OK) return st;
  const bool need = d->rows > 0;
  if (need && (x == nullptr || dy == nullptr || dx == nullptr)) return fail(GDR_EINVAL, "x, dy and dx are required");
  if (z == nullptr ? dz != nullptr : (need && dz == nullptr)) return fail(GDR_EINVAL, "gate and dgate are given together");
  const long long e = io_bytes(d->io_dtype);
  const void *io_ptrs[] = {x, dy, w, z, d_res, dx, dz};
  for (const void *p : io_ptrs)
    if (misaligned(p, e)) return fail(GDR_EINVAL, "misaligned io pointer");
  if (misaligned(dw, 4)) return fail(GDR_EINVAL, "dweight misaligned");
  const uint64_t need_ws = dw != nullptr ? bwd_ws_bytes(*d) : 0;
  if (need_ws > 0) {
    if (ws == nullptr) return fail(GDR_EINVAL, "workspace is required");
    if (ws_bytes < need_ws)
      return fail(GDR_EINVAL, "workspace_bytes = %llu, need %llu", static_cast<unsigned long long>(ws_bytes),
                  static_cast<unsigned long long>(need_ws));
    if (misaligned(ws, 256)) return fail(GDR_EINVAL, "workspace must be 256-byte aligned");
  }
  const long long D = d->D;
  const long double flat = static_cast<long double>(d->rows) * D * e;
  const Range inputs[] = {rng("x", x, span(d->rows, or_width(d->x_stride, D), D, e)),
                          rng("dy", dy, span(d->rows, or_width(d->dy_stride, D), D, e)),
                          rng("weight", w, static_cast<long double>(D) * e),
                          rng("gate", z, span(d->rows, or_width(d->gate_stride, D), D, e)),
                          rng("d_residual", d_res, span(d->rows, or_width(d->residual_stride, D), D, e))};
  const Range written[] = {rng("dx", dx, flat), rng("dweight", dw, 4.0L * D), rng("dgate", dz, flat),
                           rng("workspace", need_ws > 0 ? ws : nullptr, static_cast<long double>(need_ws))};
  return check_disjoint(written, 4, inputs, 5);
}

gdr_status_t gdr_rms_norm_bwd(const gdr_norm_desc_t *d, const void *x, const void *dy, const void *w, const void *z,
                              const void *d_res, void *dx, float *dw, void *dz, void *ws, uint64_t ws_bytes, void *stream) {
  const gdr_status_t st = gdr_validate_norm_bwd(d, x, dy, w, z, d_res, dx, dw, dz, ws, ws_bytes);
  if (st != GDR_OK) return st;
  gdr::NormArgs a{};
  a.x = x; a.dy = dy; a.w = w; a.z = z; a.res = d_res; a.dx = dx; a.dw = dw; a.dz = dz;
  a.part = dw != nullptr ? static_cast<float *>(ws) : nullptr;
  a.xs = or_width(d->x_stride, d->D); a.ds = or_width(d->dy_stride, d->D); a.zs = or_width(d->gate_stride, d->D);
  a.rs = or_width(d->residual_stride, d->D);
  a.rows = d->rows; a.D = d->D; a.eps = d->eps; a.inv_d = 1.f / d->D;
  a.groups = gdr::rms_norm_bwd_groups(d->rows, d->D, d->io_dtype);
  if (log_enabled()) std::fprintf(stderr, "[gdr] rms_norm_bwd rows=%d D=%d io=%d\n", d->rows, d->D, d->io_dtype);
  const hipError_t e = gdr::launch_rms_norm_bwd(a, d->io_dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(GDR_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"
