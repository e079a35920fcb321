// Internal declarations of the packed (variable-length, pooled-state) forms and the RMS norm:
// launch arguments, storage conversions of the three io types and wave reductions.
#pragma once

#include "common.h"

namespace gdr {

// Everything a packed launch needs, resolved and validated on the host (strides never 0).
struct PackedArgs {
  const void *q, *k, *v;
  const float *beta, *log_alpha;   // log_alpha null: no decay
  const int32_t *cu;               // null: sequence s is token s
  const int32_t *index;            // null: sequence s has slot s
  const uint8_t *has;              // null: every sequence starts from its slot
  const void *norm_w, *norm_z;
  float *pool;                     // null: start from zeros, keep nothing
  void *out;
  uint8_t *ws;                     // chunk records (gdr_packed_fwd on the matrix cores)
  long long qs, ks, vs, os, zs;    // elements between tokens
  int N, n_seqs, Hk, Hv, Dk, Dv, n_slots, qk_norm;
  float scale, qk_eps, norm_eps;
};

struct NormArgs {
  const void *x, *res, *w, *z, *dy;
  void *y, *res_out, *dx, *dz;
  float *scales, *dw, *part;       // part: [groups][D] partial sums of dw
  long long xs, rs, zs, ds;        // elements between rows of x, res, z, dy
  int rows, D, out_kind, groups;
  float eps, inv_d;                // 1 / D
};

hipError_t launch_packed_recur(const PackedArgs &a, int io_dtype, hipStream_t s);
// the norm of out's rows in place (rows of skipped sequences and of none stay as they are)
hipError_t launch_packed_norm(const PackedArgs &a, int io_dtype, hipStream_t s);
bool packed_chunk_supports(const gdr_packed_desc_t &d);
uint64_t packed_chunk_ws_bytes(const gdr_packed_desc_t &d);
hipError_t launch_packed_chunk(const PackedArgs &a, int io_dtype, hipStream_t s);
hipError_t launch_rms_norm(const NormArgs &a, int io_dtype, hipStream_t s);
int rms_norm_bwd_groups(int rows, int D, int io_dtype);
hipError_t launch_rms_norm_bwd(const NormArgs &a, int io_dtype, hipStream_t s);

// ---------------------------------------------------------------------------------
// Storage conversions: float, uint16_t (bf16 bits, common.h) and _Float16.
// ---------------------------------------------------------------------------------
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(uint16_t x) { return bf16_bits_to_f32(x); }
__device__ __forceinline__ float to_f(_Float16 x) { return static_cast<float>(x); }
template <typename IO> __device__ __forceinline__ IO from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ uint16_t from_f<uint16_t>(float x) { return f32_to_bf16_bits(x); }
template <> __device__ __forceinline__ _Float16 from_f<_Float16>(float x) { return static_cast<_Float16>(x); }

// n consecutive elements at any element alignment (gfx950 loads and stores wide words at
// addresses that are not multiples of them)
template <typename IO, int N> struct Vec {
  typedef IO type __attribute__((ext_vector_type(N), aligned(sizeof(IO))));
};
template <int N, typename IO> __device__ __forceinline__ void load_n(const IO *p, float *x) {
  const typename Vec<IO, N>::type v = *reinterpret_cast<const typename Vec<IO, N>::type *>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = to_f(static_cast<IO>(v[i]));
}
template <int N, typename IO> __device__ __forceinline__ void store_n(IO *p, const float *x) {
  typename Vec<IO, N>::type v;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = from_f<IO>(x[i]);
  *reinterpret_cast<typename Vec<IO, N>::type *>(p) = v;
}

// ---------------------------------------------------------------------------------
// Reductions; every lane gets the result, the order of the additions is fixed.
// ---------------------------------------------------------------------------------
template <int CTRL> __device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum16(float x) {   // over each 16 lanes: row rotations by 8, 4, 2, 1
  x += dpp<0x128>(x);
  x += dpp<0x124>(x);
  x += dpp<0x122>(x);
  x += dpp<0x121>(x);
  return x;
}
__device__ __forceinline__ float sum8(float x) {    // over each 8: mirrored, then within the quads
  x += dpp<0x141>(x);
  x += dpp<0xb1>(x);
  x += dpp<0x4e>(x);
  return x;
}
// max that keeps a NaN (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) { return a >= b || a != a ? a : b; }
__device__ __forceinline__ float max16(float x) {
  x = max_nan(x, dpp<0x128>(x));
  x = max_nan(x, dpp<0x124>(x));
  x = max_nan(x, dpp<0x122>(x));
  x = max_nan(x, dpp<0x121>(x));
  return x;
}
__device__ __forceinline__ float max8(float x) {
  x = max_nan(x, dpp<0x141>(x));
  x = max_nan(x, dpp<0xb1>(x));
  x = max_nan(x, dpp<0x4e>(x));
  return x;
}
template <int LANES> __device__ __forceinline__ float sum_lanes(float x) {
  x = LANES == 8 ? sum8(x) : sum16(x);
  if (LANES >= 32) x += __shfl_xor(x, 16, 64);
  if (LANES >= 64) x += __shfl_xor(x, 32, 64);
  return x;
}
template <int LANES> __device__ __forceinline__ float max_lanes(float x) {
  x = LANES == 8 ? max8(x) : max16(x);
  if (LANES >= 32) x = max_nan(x, __shfl_xor(x, 16, 64));
  if (LANES >= 64) x = max_nan(x, __shfl_xor(x, 32, 64));
  return x;
}

// 1 / sqrt(x): the hardware's approximation (2^-23 of the value) with one Newton step, which brings
// it within a rounding or two; 0 and infinite as they are, values below the normal range scaled
__device__ __forceinline__ float rsqrt_f(float x) {
  const bool tiny = x < 1.17549435e-38f;
  const float y = tiny ? x * 0x1p64f : x;
  float r = __builtin_amdgcn_rsqf(y);
  const float e = fmaf(-y * r, r, 1.f);
  r = fabsf(e) < 0.5f ? fmaf(0.5f * r, e, r) : r;   // (not where y or r is 0 or infinite)
  return tiny ? r * 0x1p32f : r;
}

// Of a gate held in IO.  The fast exponential is off by 2^-24 |z| of itself: nothing next to a 16-bit
// gate's own rounding, up to 44 roundings of an fp32 one, which takes the exact one.  0 and 1 far out.
template <typename IO> __device__ __forceinline__ float sigmoid_f(float z) {
  return __builtin_amdgcn_rcpf(1.f + (sizeof(IO) == 4 ? expf(-z) : __expf(-z)));
}
template <typename IO> __device__ __forceinline__ float silu_f(float z) { return z * sigmoid_f<IO>(z); }

// ---------------------------------------------------------------------------------
// A sequence's tokens and slot.  Device values are clamped into range, so that a bad one
// cannot reach other memory.
// ---------------------------------------------------------------------------------
__device__ __forceinline__ int clamp_tok(int x, int N) { return x < 0 ? 0 : (x > N ? N : x); }
__device__ __forceinline__ void seq_range(const PackedArgs &a, int s, int &t0, int &t1) {
  if (a.cu == nullptr) {
    t0 = s;
    t1 = s + 1;
    return;
  }
  t0 = clamp_tok(a.cu[s], a.N);
  t1 = clamp_tok(a.cu[s + 1], a.N);
  if (t1 < t0) t1 = t0;
}
// this thread's part of the search for an earlier sequence with slot idx
__device__ __forceinline__ bool seen_before(const PackedArgs &a, int s, int idx, int tid, int threads) {
  bool dup = false;
  for (int j = tid; j < s; j += threads) dup |= a.index[j] == idx;
  return dup;
}

}  // namespace gdr
