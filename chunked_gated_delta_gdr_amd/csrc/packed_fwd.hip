// The gated delta rule over packed sequences, chunked on the matrix cores (gdr_packed_fwd).
//
// Per chunk of 64 tokens, with g the cumulative log decay inside the chunk, Gamma_ij = exp(g_i - g_j),
// and every key and query written as k_i = s_i k^_i, q_i = u_i q^_i (k^, q^ scaled by powers of
// two to a fixed size; s, u hold the rest, the L2 norm included):
//     M = tril_-1(Gamma (.) k^ k^T),  T = (I + diag(beta s^2) M)^-1
//     X = beta s (.) (V - s e^g (.) (k^ S^T)),  E = T X             (E = s (.) D of the WY form)
//     O = scale u (.) (e^g (.) (q^ S^T) + tril(Gamma (.) q^ k^T) E)
//     S <- e^{g_C} S + (e^{g_C - g} (.) E)^T k^
//
// Two launches.  prep_kernel, one workgroup per (chunk, value head), all chunks at once: T, P =
// tril(Gamma (.) q^ k^T) and the row factors, as operand fragments in the workspace.  seq_kernel, per
// (sequence, value head, group of value columns): the state passes through the chunks.  A main
// wave owns 16 value columns and keeps S^T for them in its accumulators; the products chain
// S -> X -> E -> S without leaving its registers, because the accumulator layout of one 16 x 16 x 32
// product (column = lane % 16, four rows a lane group) is the B operand of the next when the A
// operand's K order is permuted to match.  Only their A operands (k^, k^T, T, the same for every wave)
// go through LDS, staged a chunk ahead by two staging waves; O is formed a chunk behind by two output
// waves, from q^ and P fragments that they load from the workspace.
//
// What bounds it (bf16, Dk = Dv = 128).  The pass through the chunks is a chain: one sequence of 32768
// tokens with 32 heads takes 870 to 930 us, some 4100 cycles a chunk, of which the main wave's 82 products
// are some 1300, its fp16 splits and the operands' way from LDS the rest; with 4 sequences of
// 4096 tokens and 16 heads (144 us, one workgroup a CU) the chain is the same and the CUs are all taken.
// The preparation moves 0.88 GB for those 32768 tokens in 250 us (3.5 TB/s): bound by its own
// arithmetic (four workgroups a CU hide its loads) and its records' way out.  Short sequences pay
// two launches and the first chunk's loads: 23 of 65 tokens on average with 8 heads 13 + 30 us.
// Tried and slower: queries through LDS with the keys (1610 us for the long sequence, their small
// scattered loads held everything up); the helpers' values in the main waves (1230 us, 1360 before);
// shuffles through LDS for the column maxima (150 cycles each).
//
// Precision.  States are as exact as fp32 makes them, in every io type: k^ and q^ are exact in fp16 (but for entries
// below 2^-21 of a key's largest), everything else on the state's path is a pair of fp16 values, 22
// bits.  The pairs need their values within fp16's range, so the wave keeps its columns under a
// power-of-two scale F per column (the recurrence is linear in each value column), set anew for
// every chunk: a pair is off by 2^-22 of the column's largest value.
// Where sizes in a column differ so much that this would show (a reset of a large state, one value far above
// the others), the chunk goes token by token in fp32 (by_token, in the main wave, 0.8 us a token); kFar below
// says when.  Asking costs a call 1 % under decays of e^-5 a chunk, 5 % under e^-10, 15 to 20 % under e^-150 (32768
// tokens: 1179, 1224 and 1340 us; unasked 1156, 1163 and 1149), fp32 up to 35 %.
// So does a chunk with an infinity or a NaN in its keys, values, gains or decays: what is not finite then
// reaches no earlier token and no other column.
// Sums are fp32, the cumulative decay is summed in 64 bits and kept as two fp32 values (its differences
// matter beside its size).
#include <type_traits>

#include "packed.h"
#include "tri_blocks.h"

namespace gdr {
namespace {

constexpr int kC = 64;     // tokens of a chunk
constexpr int kCus = 256;

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f4 mma(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// What an io type needs: parts of k^ and q^ (fp32 ones are pairs), and pairs of P, E and S in the output
// (a bf16 output rounds by 2^-9, next to which one fp16 part's 2^-12 is nothing).
template <typename IO> constexpr int kParts = sizeof(IO) == 4 ? 2 : 1;
template <typename IO> constexpr bool kExact = !std::is_same<IO, uint16_t>::value;

// One chunk's record in the workspace.  Fragments: 16 x 32 blocks (row tile mt, K block s) on and
// below the diagonal, lane l holds row 16 mt + l % 16 and the columns 32 s + 4 (l / 16) + 0..3 and
// 32 s + 16 + 4 (l / 16) + 0..3.
constexpr int kFrags = 6;
constexpr int kFragBytes = kFrags * 64 * 16;
__host__ __device__ constexpr int frag_of(int mt, int s) { return s == 0 ? mt : mt + 2; }
template <bool kPair> struct Record {
  static constexpr int T = 0;                                  // hi, lo
  // row factors [64] fp32 of the state's waves: of k^ S^T in X, of T's rows in E and in the update
  static constexpr int bk = 2 * kFragBytes, dt = bk + kC * 4, dc = dt + kC * 4;
  static constexpr int ec = dc + kC * 4;                       // e^{g_C}; how far below M a state may be to hold a size
                                                               // of 2^-kNear M (an exponent); the strongest decay
  static constexpr int staged = ec + 16;                       // what comes before goes to LDS
  // and of the others: V in X, q^ S^T and P E in O, and the factor of k^ = kf k
  static constexpr int bv = staged, oq = bv + kC * 4, op = oq + kC * 4, kf = op + kC * 4;
  static constexpr int P = kf + kC * 4;                        // hi, or hi and lo
  static constexpr int bytes = (P + (kPair ? 2 : 1) * kFragBytes + 255) / 256 * 256;
};
static_assert(Record<true>::staged % 16 == 0 && Record<true>::P % 16 == 0, "aligned fragments");
template <typename IO> using RecordOf = Record<kExact<IO>>;
// Behind the records, for every slot and key head: q^ as fragments (row tile, K block), parts next to
// each other.
template <typename IO, int DK> constexpr int kQueryBytes = 4 * (DK / 32) * kParts<IO> * 1024;

// Chunk slots: sequence s has the slots first(s) .. first(s + 1) - 1 at least for its chunks.
__device__ __forceinline__ int first_slot(const PackedArgs &a, int s) { return clamp_tok(a.cu[s], a.N) / kC + s; }

// row i, 16-byte chunk q of an LDS tile with rows of ROW bytes: chunks permuted so that the 16
// rows of a fragment lie in different banks
// (and, with short rows, the rows 8 apart that a staging wave writes at once)
template <int ROW> __device__ __forceinline__ int swz(int i, int q) {
  return i * ROW + ((ROW == 128 ? q ^ (((i >> 1) + (i >> 4)) & 7) : q ^ (i & 15)) << 4);
}

// 2^n for n in the normal range
__device__ __forceinline__ float pow2(int n) { return __int_as_float((n + 127) << 23); }
constexpr float kInf = __builtin_inff(), kNaN = __builtin_nanf("");
// n with 2^n <= x < 2^(n + 1) (-127 below the normal range); kNone for zero, infinite and NaN
constexpr int kNone = -1000;
__device__ __forceinline__ int log2_floor(float x) {
  return x > 0.f && x < kInf ? static_cast<int>(__float_as_uint(x) >> 23) - 127 : kNone;
}
// the same, at least -100, 0 where there is none: for factors whose inverse is needed too
__device__ __forceinline__ int log2_near(float x) {
  const int e = log2_floor(x);
  return e == kNone ? 0 : max(-100, e);
}

// Where fp16 operands are put.  fp16's smallest step is 2^-24, so a pair has its 22 bits for values
// from 2^-2 on, and an operand's largest value has to lie well above:
// the columns of S and V at 2^kTop and T's rows as well, key rows at 2^7, query rows at 2^3 (their
// products, 128 of them, come to 2^19 at most: P is kept 2^-5 of itself).
// A unit key's s is then about 2^-9 and so are X and E beside V and S: they are kept 2^kLift times
// larger, and with them the accumulators of S, which are brought down again where they are split.
// X and E may be some 2^5 larger than S and V (the size of sums of 128 products) and stay in range.
constexpr int kTop = 9, kKeyTop = 7, kQueryTop = 3, kPShift = 5, kLift = 9;
constexpr int kDepth = 12;   // operands under way from LDS (at most 15 reads are counted)
constexpr int kMaxScale = 110;
constexpr float kOver = 32768.f;

// What one scale for a column's 64 tokens and state costs.  With M the largest of them, fp16's smallest
// step leaves X, E, S and T's products off by 2^-34 M, and P's products with E by 2^-30 of the largest up
// to the row; a state or rows whose own size has fallen far below M, by a reset or strong decays or
// because M comes later, would lose their bits to that.  So the sizes are followed through the chunk,
//     A_i = max(alpha_i A_{i-1}, |bv_i V_i|)   from A_-1 = |S|   (the rule's, without what it erases).
// Far is A_63 < 2^-14 M (else states are good to 2^-20, beside fp32's own roundings of a chunk), and A_i < 2^-kFar M
// or < 2^-kFarBefore of the largest up to i (else rows to 2^-12 in bf16, as the output's one-part factors, 2^-13
// in fp16 and 2^-18 in fp32).  The chunk goes token by token where two rows running are far in a column, or
// where a column's M makes a row far as measured by the row's largest of 16 columns (one small value among
// its neighbours, of which random data always has some, is neither).
constexpr int kFarEnd = 14;
template <typename IO> constexpr int kFar = sizeof(IO) == 4 ? 16 : kExact<IO> ? 21 : 22;
template <typename IO> constexpr int kFarBefore = sizeof(IO) == 4 ? 12 : kExact<IO> ? 17 : 18;
template <typename IO> constexpr int kNear = kFarEnd < kFarBefore<IO> ? kFarEnd : kFarBefore<IO>;   // near enough for all three

// hi + lo = x to 22 bits, for two values: one conversion and two mixed-precision multiply-adds.  x and
// hi are made opaque: were the product behind x contracted into hi's conversion in one place and
// not in the other, hi and its rest would belong to different roundings (and left to itself the
// compiler converts twice).  one is an opaque 1, without which the multiply-adds fall apart.
__device__ __forceinline__ float opaque(float x) {
  asm("" : "+s"(x));
  return x;
}
__device__ __forceinline__ void split2(float x, float y, float one, h2 &hi, h2 &lo) {
  asm("" : "+v"(x), "+v"(y));
  uint32_t u = __builtin_bit_cast(uint32_t, h2{static_cast<_Float16>(x), static_cast<_Float16>(y)});
  asm("" : "+v"(u));
  hi = __builtin_bit_cast(h2, u);
  lo = h2{static_cast<_Float16>(fmaf(x, one, -static_cast<float>(hi[0]))),
          static_cast<_Float16>(fmaf(y, one, -static_cast<float>(hi[1])))};
}
__device__ __forceinline__ void split8(f4 x, f4 y, float one, h8 &hi, h8 &lo) {
  h2 u[4], v[4];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    split2(x[2 * e], x[2 * e + 1], one, u[e], v[e]);
    split2(y[2 * e], y[2 * e + 1], one, u[e + 2], v[e + 2]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    hi[e] = u[e / 2][e & 1];
    lo[e] = v[e / 2][e & 1];
  }
}
__device__ __forceinline__ void split(float x, _Float16 &hi, _Float16 &lo) {
  asm("" : "+v"(x));
  hi = static_cast<_Float16>(x);
  lo = static_cast<_Float16>(x - static_cast<float>(hi));
}

// Rows of a chunk through a buffer descriptor: reads behind its last row give zeros, writes there
// are dropped.  Offsets are 32 bits: 64 rows of at most 2^23 elements.
template <typename IO> struct Rows {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Rows(const IO *p, int n, long long stride, int width)
      : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<IO *>(p), 0,
                                            static_cast<int>(n > 0 ? ((n - 1) * stride + width) * sizeof(IO) : 0), 0x00020000)) {}
  typedef IO io8 __attribute__((ext_vector_type(8)));
  __device__ __forceinline__ io8 get8(uint32_t at) const {   // at any alignment
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    typedef IO half __attribute__((ext_vector_type(16 / sizeof(IO))));
    if constexpr (sizeof(IO) == 4) {
      const half x = __builtin_bit_cast(half, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
      const half y = __builtin_bit_cast(half, __builtin_amdgcn_raw_buffer_load_b128(r, at + 16, 0, 0));
      return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      return __builtin_bit_cast(io8, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
    }
  }
  __device__ __forceinline__ f4 get4(uint32_t at) const {   // four words
    return __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
  }
  __device__ __forceinline__ float get1(uint32_t at) const {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
  }
  __device__ __forceinline__ void put4(f4 x, uint32_t at) const {   // four columns, at any alignment
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    if constexpr (sizeof(IO) == 4) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, x), r, at, 0, 0);
    } else {
      typedef IO io4 __attribute__((ext_vector_type(4)));
      const io4 y = {from_f<IO>(x[0]), from_f<IO>(x[1]), from_f<IO>(x[2]), from_f<IO>(x[3])};
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, y), r, at, 0, 0);
    }
  }
};

// x[e] of lane 4 a + b becomes x[b] of lane 4 a + e
__device__ __forceinline__ f4 quad_transpose(f4 x, int lane) {
  const bool odd = lane & 1, high = lane & 2;
  // lanes 1 apart exchange their off-diagonal entries of the 2 x 2 blocks, lanes 2 apart the blocks
  const float p = dpp<0xb1>(odd ? x[0] : x[1]), q = dpp<0xb1>(odd ? x[2] : x[3]);
  x = odd ? f4{p, x[1], q, x[3]} : f4{x[0], p, x[2], q};
  const float u = dpp<0x4e>(high ? x[0] : x[2]), v = dpp<0x4e>(high ? x[1] : x[3]);
  return high ? f4{u, v, x[2], x[3]} : f4{x[0], x[1], u, v};
}

// ------------------------------------------------------------------------------------------
// Chunk-parallel preparation
// ------------------------------------------------------------------------------------------
// x[lane] <- x[0] + .. + x[lane], by row shifts and broadcasts
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_add(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<uint32_t>(u), CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<uint32_t>(u >> 32), CTRL, ROWS, 0xf, false);
  return x + __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double scan64(double x) {
  x = dpp_add<0x111, 0xf>(x);   // from 1, 2, 4 and 8 lanes back in the rows of 16
  x = dpp_add<0x112, 0xf>(x);
  x = dpp_add<0x114, 0xf>(x);
  x = dpp_add<0x118, 0xf>(x);
  x = dpp_add<0x142, 0xa>(x);   // rows 1 and 3 from the end of rows 0 and 2
  return dpp_add<0x143, 0xc>(x);   // rows 2 and 3 from the end of row 1
}

// over the four lanes of a column: swapping the register with itself puts each lane next to its
// neighbour 16 (32) lanes on (a shuffle through LDS takes 150 cycles, this a few)
__device__ __forceinline__ float max_col(float m) {
  uint32_t u = __float_as_uint(m);
  auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  m = __builtin_elementwise_maximum(__uint_as_float(p[0]), __uint_as_float(p[1]));
  u = __float_as_uint(m);
  p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_elementwise_maximum(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float min_col(float m) { return -max_col(-m); }

// LDS: k^ and q^ are dead once M and P are formed, L and T take their place (four workgroups a CU
// for 16-bit types, which hides the loads and the inverse's chain of small products).
template <typename IO, int DK> struct PrepLds {
  static constexpr int LD = 68;                              // L and T rows, 16-byte aligned
  static constexpr int part = kC * DK * 2, Q = kParts<IO> * part, T = kC * LD * 4;
  static constexpr int big = 2 * Q > 2 * T ? 2 * Q : 2 * T;
};

template <typename IO, int DK>
__global__ __launch_bounds__(256) void prep_kernel(PackedArgs a) {
  using Rec = RecordOf<IO>;
  using Lds = PrepLds<IO, DK>;
  constexpr int ROW = DK * 2, LD = Lds::LD, NP = kParts<IO>, PART = Lds::part, NS = DK / 32;
  __shared__ __align__(16) uint8_t big[Lds::big];
  __shared__ __align__(16) float Zs[32][36];
  __shared__ float sk[kC], su[kC], bt[kC];
  __shared__ __align__(16) float gh[kC], gl[kC];   // cumulative log decay, to 48 bits
  uint8_t *Ks = big, *Qs = big + Lds::Q;
  float(*L)[LD] = reinterpret_cast<float(*)[LD]>(big);
  float(*Tm)[LD] = reinterpret_cast<float(*)[LD]>(big + Lds::T);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  const int h = blockIdx.x % a.Hv, slot = blockIdx.x / a.Hv, hk = h / (a.Hv / a.Hk);
  int s = -1;   // the last sequence whose slots begin at or before this one
  for (int step = (a.n_seqs - 1) / 256 + 1;; step = 1) {   // every step-th of the next 256 step, then each
    const int at = max(s, 0) + (s < 0 ? tid : tid + 1) * step;
    const int found = __syncthreads_count(at < a.n_seqs && first_slot(a, at) <= slot);
    s = s < 0 ? (found - 1) * step : s + found;
    if (step == 1 || s < 0) break;
  }
  if (s < 0) return;
  int t0, t1;
  seq_range(a, s, t0, t1);
  const int first = first_slot(a, s);
  t0 += (slot - first) * kC;
  const int n = min(kC, t1 - t0);
  if (slot < first || n <= 0) return;
  if (a.index != nullptr && a.index[s] < 0) return;

  uint8_t *rec = a.ws + (static_cast<long long>(slot) * a.Hv + h) * Rec::bytes;
  // rows, 16 lanes a row: all loads first (rows past the end read the last one and count as zeros)
  constexpr int E = DK / 16;   // entries of a lane
  typedef typename Vec<IO, E>::type raw;
  const IO *kp = static_cast<const IO *>(a.k) + static_cast<long long>(hk) * a.Dk + t0 * a.ks;
  const IO *qp = static_cast<const IO *>(a.q) + static_cast<long long>(hk) * a.Dk + t0 * a.qs;
  const int c0 = (tid & 15) * E;
  const bool chan = c0 < a.Dk;   // (channels from Dk on are zeros)
  const bool whole = n == kC && a.Dk == DK;
  raw rows[2][4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t i = min(16 * p + (tid >> 4), n - 1);
    rows[0][p] = *reinterpret_cast<const raw *>(kp + (i * static_cast<uint32_t>(a.ks) + (chan ? c0 : 0)));
    rows[1][p] = *reinterpret_cast<const raw *>(qp + (i * static_cast<uint32_t>(a.qs) + (chan ? c0 : 0)));
  }
  float drop = 0.f;   // (wave 0) the strongest log decay
  if (wave == 0) {   // cumulative log decay and the gains; tokens past the end change nothing
    const long long at = static_cast<long long>(t0 + min(lane, n - 1)) * a.Hv + h;
    float la = a.log_alpha != nullptr ? a.log_alpha[at] : 0.f;
    const float b = a.beta[at];
    if (la < -200.f) la = -200.f;   // exp(-200) is zero in fp32: keeps the differences finite
    const double x = scan64(lane < n ? la : 0.f);
    gh[lane] = static_cast<float>(x);
    gl[lane] = static_cast<float>(x - gh[lane]);
    bt[lane] = lane < n ? (la < kInf ? b : kNaN) : 0.f;
    drop = fminf(lane < n ? la : 0.f, 0.f);
    drop = fminf(drop, dpp<0x128>(drop));
    drop = fminf(drop, dpp<0x124>(drop));
    drop = fminf(drop, dpp<0x122>(drop));
    drop = min_col(fminf(drop, dpp<0x121>(drop)));
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int i = 16 * p + (tid >> 4);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float x[E], m = 0.f, ss = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = to_f(static_cast<IO>(rows[which][p][e]));
      if (!whole && !(i < n && chan)) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) m = __builtin_elementwise_maximum(m, fabsf(x[e]));
      m = __builtin_elementwise_maximum(m, dpp<0x128>(m));
      m = __builtin_elementwise_maximum(m, dpp<0x124>(m));
      m = __builtin_elementwise_maximum(m, dpp<0x122>(m));
      m = __builtin_elementwise_maximum(m, dpp<0x121>(m));
      const int ex = log2_near(m) - (which == 0 ? kKeyTop : kQueryTop);
      const float f = pow2(-ex);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] *= f;
      float rest = pow2(ex);
      if (a.qk_norm) {   // |k|^2 = 2^(2 ex) sum k^2: 1 / sqrt(|k|^2 + eps) = 2^-ex / sqrt(sum + 2^(-2 ex) eps)
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
        ss = sum16(ss);
        const float eps = a.qk_eps * f * f;
        // (a row so far below eps that eps leaves the type on the row's scale: 2^-ex / sqrt(2^(-2 ex) eps) = 1 / sqrt(eps))
        rest = eps < kInf ? rsqrt_f(ss + eps) : rsqrt_f(a.qk_eps) * rest;
        if (ss == 0.f && a.qk_eps == 0.f) rest = kNaN;   // 0 / 0
      }
      typedef _Float16 hE __attribute__((ext_vector_type(E)));
      uint8_t *dst = (which == 0 ? Ks : Qs) + swz<ROW>(i, c0 / 8) + (c0 % 8) * 2;
      hE y, z;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        _Float16 hi, lo;
        split(x[e], hi, lo);
        y[e] = hi;
        z[e] = lo;
      }
      *reinterpret_cast<hE *>(dst) = y;
      if constexpr (NP == 2) *reinterpret_cast<hE *>(dst + PART) = z;
      if (which == 0 && !(m < kInf)) rest = kNaN;   // (a mark, as the values' factor: see by_token)
      if ((tid & 15) == 0) {
        // (past the end rows of zeros stand in, whose norm without eps is 1 / 0: they weigh nothing)
        (which == 0 ? sk : su)[i] = i < n ? rest : 0.f;
        // (the state's pass reads a row in the place of those past the end)
        if (which == 0) reinterpret_cast<float *>(rec + Rec::kf)[i] = i < n ? f : 0.f;
      }
    }
  }
  __syncthreads();

  // M^T and P^T tiles: wave w has the columns i = 16 w + r and every row tile j <= w.  The
  // accumulators then hold rows of M and P, four columns a lane group: P's fragments as they are
  const int i = 16 * wave + r;
  f4 m[4], p[4];
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) m[jt] = p[jt] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    h8 kb[NP], qb[NP];
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      kb[u] = *reinterpret_cast<const h8 *>(Ks + u * PART + swz<ROW>(i, 4 * k + g));
      qb[u] = *reinterpret_cast<const h8 *>(Qs + u * PART + swz<ROW>(i, 4 * k + g));
    }
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      if (jt > wave) continue;
      const uint8_t *at = Ks + swz<ROW>(16 * jt + r, 4 * k + g);
      const h8 ka = *reinterpret_cast<const h8 *>(at);
      if constexpr (NP == 2) {
        const h8 kl = *reinterpret_cast<const h8 *>(at + PART);
        m[jt] = mma(kl, kb[0], m[jt]);
        m[jt] = mma(ka, kb[1], m[jt]);
        p[jt] = mma(kl, qb[0], p[jt]);
        p[jt] = mma(ka, qb[1], p[jt]);
      }
      m[jt] = mma(ka, kb[0], m[jt]);
      p[jt] = mma(ka, qb[0], p[jt]);
    }
  }
  if (h % (a.Hv / a.Hk) == 0) {   // q^ for the output waves, once a key head: channels in the state's K order
    const long long slots = a.N / kC + a.n_seqs;
    uint8_t *dst = a.ws + slots * a.Hv * Rec::bytes + (static_cast<long long>(slot) * a.Hk + hk) * kQueryBytes<IO, DK> + lane * 16;
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        const uint8_t *src = Qs + u * PART + 8 * (g & 1);
        const h4 lo = *reinterpret_cast<const h4 *>(src + swz<ROW>(i, 4 * k + (g >> 1)));
        const h4 hi = *reinterpret_cast<const h4 *>(src + swz<ROW>(i, 4 * k + 2 + (g >> 1)));
        *reinterpret_cast<h8 *>(dst + ((wave * NS + k) * NP + u) * 1024) = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
  }
  __syncthreads();   // k^ and q^ are read
  if (tid == 0) Tm[0][64] = __expf(drop);   // (beside T: its rows are padded)
  const float gi = gh[i], gi_low = gl[i];
  const float si = sk[i], bs = bt[i] * si * si;
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    f4 l = {0.f, 0.f, 0.f, 0.f};
    if (jt <= wave) {
      const f4 gj = *reinterpret_cast<const f4 *>(&gh[16 * jt + 4 * g]), gj_low = *reinterpret_cast<const f4 *>(&gl[16 * jt + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 16 * jt + 4 * g + e;
        // (off by 2^-24 of 1 at most, however large the exponent: it is never positive)
        const float gam = __expf((gi - gj[e]) + (gi_low - gj_low[e]));
        if (j < i) l[e] = bs * (gam * m[jt][e]);
        p[jt][e] = j <= i ? gam * (p[jt][e] * pow2(-kPShift)) : 0.f;
      }
    } else {
      *reinterpret_cast<f4 *>(&Tm[i][16 * jt + 4 * g]) = l;   // blocks above the diagonal
    }
    *reinterpret_cast<f4 *>(&L[i][16 * jt + 4 * g]) = l;
  }
#pragma unroll
  for (int s2 = 0; s2 < 2; ++s2) {   // P's fragments
    if (s2 <= wave / 2) {
      h8 hi, lo;
      split8(p[2 * s2], p[2 * s2 + 1], opaque(1.f), hi, lo);
      uint8_t *dst = rec + Rec::P + (frag_of(wave, s2) * 64 + lane) * 16;
      *reinterpret_cast<h8 *>(dst) = hi;
      if constexpr (kExact<IO>) *reinterpret_cast<h8 *>(dst + kFragBytes) = lo;
    }
  }
  __syncthreads();
  tri::inverse_blocks<LD, LD>(L, Tm, Zs, -1, tid);
  {   // T's fragments, each row under a power of two, and the row factors
    f4 x[4];
    float top = 0.f;
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      x[jt] = *reinterpret_cast<const f4 *>(&Tm[i][16 * jt + 4 * g]);
#pragma unroll
      for (int e = 0; e < 4; ++e) top = __builtin_elementwise_maximum(top, fabsf(x[jt][e]));
    }
    top = __builtin_elementwise_maximum(top, __shfl_xor(top, 16, 64));
    top = __builtin_elementwise_maximum(top, __shfl_xor(top, 32, 64));
    const int ex = log2_near(top) - kTop;
    const float f = pow2(-ex);
#pragma unroll
    for (int s2 = 0; s2 < 2; ++s2) {
      if (s2 <= wave / 2) {
        h8 hi, lo;
        split8(x[2 * s2] * f, x[2 * s2 + 1] * f, opaque(1.f), hi, lo);
        uint8_t *dst = rec + Rec::T + (frag_of(wave, s2) * 64 + lane) * 16;
        *reinterpret_cast<h8 *>(dst) = hi;
        *reinterpret_cast<h8 *>(dst + kFragBytes) = lo;
      }
    }
    if (g == 0) {
      const auto put = [&](int at, float x) { reinterpret_cast<float *>(rec + at)[i] = x; };
      const float tau = pow2(ex), eg = expf(gi), ec = expf((gh[kC - 1] - gi) + (gl[kC - 1] - gi_low));
      put(Rec::bv, top < kInf ? bt[i] * si * pow2(kLift) : kNaN);
      put(Rec::bk, -bs * eg * pow2(kLift));
      put(Rec::dt, tau);
      put(Rec::dc, tau * ec);
      put(Rec::oq, a.scale * su[i] * eg);
      put(Rec::op, a.scale * su[i] * pow2(kPShift - kLift));
      if (i == kC - 1) *reinterpret_cast<f4 *>(rec + Rec::ec) = f4{eg, __int_as_float(kNear<IO> - 1 - static_cast<int>(ceilf(-1.442695f * gi))), Tm[0][64], 0.f};
    }
  }
}

// ------------------------------------------------------------------------------------------
// The state's pass
// ------------------------------------------------------------------------------------------

// A workgroup: MAIN main waves of 16 value columns each, which carry the state; two staging waves, which
// bring the next chunk's keys, values, T and row factors to LDS; as many output waves as main ones,
// which, a chunk behind, form O from the fp16 parts of S and E that the main waves leave in LDS and
// from queries and P, which they load themselves.  Main waves have a SIMD each, 0 and 1, the others
// sit on the rest (waves go to the SIMDs in turn; those without a role end at once).
//
// Two main waves, or one where that leaves no more workgroups than CUs: the 32768-token sequence of 32
// heads takes 857 us with one (each CU's LDS serves one main wave), 907 with two; 4 x 4096 tokens
// of 16 heads 241 and 140, 23 short sequences 48 and 30, where the CUs are taken already.
constexpr int kStaging = 2, kFirstStaging = 2, kWaves = 8;
constexpr int first_out(int main) { return main == 1 ? 5 : 6; }

template <typename IO, int DK, int MAIN> struct Lds {
  using Rec = RecordOf<IO>;
  static constexpr int NP = kParts<IO>, NE = kExact<IO> ? 2 : 1, NS = DK / 32;
  // a stage: one chunk's operands
  static constexpr int part = kC * DK * 2;
  static constexpr int K = 0;                       // k^ [64][DK], channels permuted to the state's K order
  static constexpr int KT = NP * part;              // k^T [DK][64], tokens permuted likewise
  static constexpr int rec = 2 * NP * part;         // the record's first part
  static constexpr int cols = 16 * MAIN;            // value columns
  static constexpr int V = rec + Rec::staged;       // bv V [column][64 rows, padded]
  static constexpr int v_col = 68;                  // (columns 4 banks apart)
  static constexpr int stage = V + cols * v_col * 4;
  // a main wave's hand-over, twice: S by K block, E by K block, parts next to each other, as B operands;
  // then the columns' factors: how far S was brought down since, and 1 / F (0: the chunk is written already)
  static constexpr int E = NS * NE * 1024, scale = E + 2 * NE * 1024, hand = scale + 2 * 16 * 4;
  static constexpr int hands = 2 * MAIN * hand;
  // two stages where they fit beside each other: the next chunk is written during this one
  static constexpr int room = 160 * 1024 - 512;
  static constexpr int stages = 2 * stage + hands <= room ? 2 : 1;
  static constexpr int out = stages * stage, bytes = out + hands;
  static_assert(bytes <= room && stage % 16 == 0 && hand % 16 == 0, "a workgroup's LDS");
};

// The barriers of a chunk, alike for every role: after the first, stage c is filled and chunk c - 1
// done.  With one stage two: chunk c - 1 done, then stage c filled.
template <int kStages> __device__ __forceinline__ void chunk_done(int c) {
  if (kStages == 1 && c > 0) __syncthreads();
}

// The keys of a stage.
template <typename IO, int DK> struct Keys {
  using L = Lds<IO, DK, 1>;   // (the same up to the values)
  using Rec = RecordOf<IO>;
  static constexpr int kThreads = 64 * kStaging;
  static constexpr int kBlocks = 16 * (DK / 8) / kThreads;   // 4 tokens x 8 channels, of each lane
  static_assert(kBlocks * kThreads == 16 * (DK / 8), "whole blocks");
  typename Rows<IO>::io8 k[kBlocks][4];
  f4 kf[kBlocks];

  __device__ __forceinline__ void load(const Rows<IO> &rows, uint32_t stride, int Dk, const uint8_t *rec, int hl) {
    const Rows<float> record(reinterpret_cast<const float *>(rec), 1, 0, Rec::P / 4);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int blk = hl + b * kThreads, cg = blk % (DK / 8), tg = blk / (DK / 8);
      kf[b] = record.get4(Rec::kf + 16 * tg);
#pragma unroll
      for (int e = 0; e < 4; ++e)   // (channels from Dk on: no such offset, zeros)
        k[b][e] = rows.get8(8 * cg < Dk ? ((4 * tg + e) * stride + 8 * cg) * static_cast<uint32_t>(sizeof(IO)) : 0x80000000u);
    }
  }

  __device__ __forceinline__ void store(uint8_t *st, int hl) const {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int blk = hl + b * kThreads, cg = blk % (DK / 8), tg = blk / (DK / 8);
      // channels 8 cg + 0..3 and + 4..7: K block cg / 4, groups gc, gc + 1, half hc
      const int gc = (2 * cg) & 3, hc = (cg >> 1) & 1, qc = 4 * (cg >> 2) + gc;
      // pairs of channels 8 cg + 2 c, 2 c + 1 of token 4 tg + e
      h2 x[L::NP][4][4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float u = to_f(static_cast<IO>(k[b][e][2 * c])) * kf[b][e], w = to_f(static_cast<IO>(k[b][e][2 * c + 1])) * kf[b][e];
          if constexpr (L::NP == 2)
            split2(u, w, opaque(1.f), x[0][e][c], x[1][e][c]);
          else
            x[0][e][c] = h2{static_cast<_Float16>(u), static_cast<_Float16>(w)};
        }
#pragma unroll
      for (int p = 0; p < L::NP; ++p) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<h4 *>(st + L::K + p * L::part + swz<DK * 2>(4 * tg + e, qc + u) + 8 * hc) =
                __builtin_shufflevector(x[p][e][2 * u], x[p][e][2 * u + 1], 0, 1, 2, 3);
        // tokens 4 tg + 0..3 of a channel's row: K block tg / 8, group tg % 4, half (tg / 4) % 2
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t r0 = __builtin_bit_cast(uint32_t, x[p][0][c]), r1 = __builtin_bit_cast(uint32_t, x[p][1][c]);
          const uint32_t r2 = __builtin_bit_cast(uint32_t, x[p][2][c]), r3 = __builtin_bit_cast(uint32_t, x[p][3][c]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t sel = u == 0 ? 0x05040100u : 0x07060302u;   // the low or the high halves
            typedef uint32_t u2 __attribute__((ext_vector_type(2)));
            *reinterpret_cast<u2 *>(st + L::KT + p * L::part + swz<128>(8 * cg + 2 * c + u, 4 * (tg >> 3) + (tg & 3)) +
                                    8 * ((tg >> 2) & 1)) =
                u2{__builtin_amdgcn_perm(r1, r0, sel), __builtin_amdgcn_perm(r3, r2, sel)};
          }
        }
      }
    }
  }
};

// The values (as bv V) of a stage, and the record's first part.
template <typename IO, int DK, int MAIN> struct Values {
  using L = Lds<IO, DK, MAIN>;
  using Rec = RecordOf<IO>;
  static constexpr int kCols = L::cols, kThreads = 64 * kStaging;
  static constexpr int kItems = kC * kCols / 8 / kThreads;   // 1 token x 8 value columns
  static constexpr int kWords = (Rec::staged / 16 + kThreads - 1) / kThreads;
  static_assert(kItems * kThreads * 8 == kC * kCols, "whole blocks");
  typename Rows<IO>::io8 v[kItems];
  float bv[kItems];
  f4 words[kWords];

  __device__ __forceinline__ void load(const Rows<IO> &rows, uint32_t stride, int cols, const uint8_t *rec, int hl) {
    const Rows<float> record(reinterpret_cast<const float *>(rec), 1, 0, Rec::P / 4);
#pragma unroll
    for (int b = 0; b < kItems; ++b) {
      const int item = hl + b * kThreads, cg = item % (kCols / 8), i = item / (kCols / 8);
      bv[b] = record.get1(Rec::bv + 4 * i);
      v[b] = rows.get8((i * stride + min(8 * cg, cols - 8)) * sizeof(IO));
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) words[w] = record.get4(16 * (hl + w * kThreads));
  }

  __device__ __forceinline__ void store(uint8_t *st, int hl) const {
#pragma unroll
    for (int b = 0; b < kItems; ++b) {
      const int item = hl + b * kThreads, cg = item % (kCols / 8), i = item / (kCols / 8);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<float *>(st + L::V + ((8 * cg + c) * L::v_col + i) * 4) = to_f(static_cast<IO>(v[b][c])) * bv[b];
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const int at = hl + w * kThreads;
      if (at * 16 < Rec::staged) *reinterpret_cast<f4 *>(st + L::rec + 16 * at) = words[w];
    }
  }
};

// Output: O = oq (q^ S^T) + op (P E) of a chunk for 16 value columns.
template <typename IO, int DK> struct Output {
  using L = Lds<IO, DK, 1>;   // (a hand-over is the same)
  using Rec = RecordOf<IO>;
  static constexpr int NS = L::NS, NP = L::NP, NE = L::NE;
  // a period ahead where the registers hold it (fp32 queries, which are pairs, and the row factors
  // beside pairs of P are read when they are used)
  static constexpr bool kAhead = NP == 1, kRowsAhead = NE == 1;
  h8 q[kAhead ? 4 * NS : 1], p[kFrags * NE];
  f4 oq[kRowsAhead ? 4 : 1], op[kRowsAhead ? 4 : 1];
  const uint8_t *qat, *rows;   // of this lane

  __device__ __forceinline__ void load(const uint8_t *qp, const uint8_t *rec, int lane) {
    qat = qp + lane * 16;
    rows = rec + 16 * (lane >> 4);
    if constexpr (kAhead) {
#pragma unroll
      for (int j = 0; j < 4 * NS; ++j) q[j] = *reinterpret_cast<const h8 *>(qat + j * 1024);
    }
#pragma unroll
    for (int j = 0; j < kFrags * NE; ++j)
      p[j] = *reinterpret_cast<const h8 *>(rec + Rec::P + (j % NE * kFragBytes + (j / NE * 64 + lane) * 16));
    if constexpr (kRowsAhead) {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        oq[mt] = row(Rec::oq, mt);
        op[mt] = row(Rec::op, mt);
      }
    }
  }
  __device__ __forceinline__ f4 row(int at, int mt) const { return *reinterpret_cast<const f4 *>(rows + at + 64 * mt); }

  // q^ S^T
  __device__ __forceinline__ void query(const uint8_t *hand, int lane, f4 *x) const {
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) x[mt] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      h8 s[NE];
#pragma unroll
      for (int u = 0; u < NE; ++u) s[u] = *reinterpret_cast<const h8 *>(hand + ((k * NE + u) * 64 + lane) * 16);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        const int j = (mt * NS + k) * NP;
        h8 hi;
        if constexpr (kAhead) {
          hi = q[j];
        } else {
          hi = *reinterpret_cast<const h8 *>(qat + j * 1024);
          x[mt] = mma(*reinterpret_cast<const h8 *>(qat + (j + 1) * 1024), s[0], x[mt]);
        }
        if constexpr (NE == 2) x[mt] = mma(hi, s[1], x[mt]);
        x[mt] = mma(hi, s[0], x[mt]);
      }
    }
  }
  // returns 1 / F
  __device__ __forceinline__ float values(const uint8_t *hand, int lane, const f4 *x, f4 *o) const {
    f4 pe[4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) pe[mt] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      h8 e[NE];
#pragma unroll
      for (int u = 0; u < NE; ++u) e[u] = *reinterpret_cast<const h8 *>(hand + L::E + ((k * NE + u) * 64 + lane) * 16);
#pragma unroll
      for (int mt = 2 * k; mt < 4; ++mt) {
        const int f = frag_of(mt, k) * NE;
        if constexpr (NE == 2) {
          pe[mt] = mma(p[f + 1], e[0], pe[mt]);
          pe[mt] = mma(p[f], e[1], pe[mt]);
        }
        pe[mt] = mma(p[f], e[0], pe[mt]);
      }
    }
    const float *scale = reinterpret_cast<const float *>(hand + L::scale) + (lane & 15);
    const float down = scale[0], Finv = scale[16];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      const f4 u = kRowsAhead ? oq[kRowsAhead ? mt : 0] : row(Rec::oq, mt), w = kRowsAhead ? op[kRowsAhead ? mt : 0] : row(Rec::op, mt);
      o[mt] = (u * (x[mt] * down) + w * pe[mt]) * Finv;
    }
    return Finv;
  }
};

// largest magnitude (NaN if there is one: three operands an instruction, none of them quieted first)
__device__ __forceinline__ float max4(float m, f4 x) {
  m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(x[0])), fabsf(x[1]));
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(x[2])), fabsf(x[3]));
}
__device__ __forceinline__ float sum_col(float x) {
  uint32_t u = __float_as_uint(x);
  auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  u = __float_as_uint(__uint_as_float(p[0]) + __uint_as_float(p[1]));
  p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Whether no size falls too far below the column's M, looked at closer: its state holds it up alone, or each
// pair of rows has one that carries the next pair (with the state, for the first), or each row holds its own;
// rows from n on left out.  v: the column's 64 values bv V; s: its state's size; decay: the chunk's; decay3: no
// decay over three tokens is below it.
template <typename IO>
__device__ __forceinline__ bool clearly_near(const float *v, float s, float M, float decay, float decay3, int n, int g) {
  float pairs = kInf, each = kInf, last = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f4 x = *reinterpret_cast<const f4 *>(v + 16 * g + 4 * j);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * g + 4 * j + e;   // (rows from n on: as if there were none)
      if ((e & 1) == 0) pairs = i < n ? fminf(pairs, fmaxf(fmaxf(fabsf(x[e]), fabsf(x[e + 1])), i == 0 ? s : 0.f)) : pairs;
      each = i < n ? fminf(each, fabsf(x[e])) : each;
      last = i == n - 1 ? fabsf(x[e]) : last;
      if (j == 0 && e == 0) pairs = g == 0 ? fminf(pairs, fmaxf(fabsf(x[0]), s)) : pairs;
    }
  }
  pairs = min_col(pairs);
  each = min_col(each);
  last = max_col(last);
  return !(pairs * decay3 < M * pow2(-kNear<IO>)) || !(each < M * pow2(-kFarBefore<IO>) || last < M * pow2(-kFarEnd)) ||
         !(s * decay < M * pow2(-kNear<IO>));
}

// Whether the chunk is far, from the sizes themselves: each lane follows 16 rows from nothing, then from what
// the lanes before leave.
template <typename IO, typename Args>
__device__ __forceinline__ bool falls_far(const Args &a, const float *v, float s, float M, int t0, int n, int h, int lane) {
  const int g = lane >> 4;
  float x[16], al[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int i = 16 * g + j;
    x[j] = fabsf(v[i]);
    al[j] = a.log_alpha != nullptr && i < n ? a.log_alpha[static_cast<long long>(t0 + i) * a.Hv + h] : 0.f;
  }
  float A = 0.f, P = 1.f, m = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    al[j] = __expf(al[j]);
    A = fmaxf(A * al[j], x[j]);
    P *= al[j];
    m = fmaxf(m, x[j]);
  }
  float size = s, most = s;
#pragma unroll
  for (int b = 0; b < 3; ++b) {
    const int from = (lane & 15) + 16 * b;
    const float Ab = __shfl(A, from, 64), Pb = __shfl(P, from, 64), mb = __shfl(m, from, 64);
    if (b < g) {
      size = fmaxf(size * Pb, Ab);
      most = fmaxf(most, mb);
    }
  }
  const auto far_below = [&](float a, float end) {   // (0: nothing there to lose)
    return a > 0.f && (a < M * pow2(-kFar<IO>) || a < most * pow2(-kFarBefore<IO>) || a < end);
  };
  bool far = false, before = far_below(size, 0.f);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    size = fmaxf(size * al[j], x[j]);
    most = fmaxf(most, x[j]);
    float row = fmaxf(size, dpp<0x128>(size));
    row = fmaxf(row, dpp<0x124>(row));
    row = fmaxf(row, dpp<0x122>(row));
    row = fmaxf(row, dpp<0x121>(row));
    const float end = j == 15 && g == 3 ? M * pow2(-kFarEnd) : 0.f;
    const bool here = far_below(size, end);
    far |= (here && before) || far_below(row, end);
    before = here;
    if (j == 14 && g == 3) before |= far_below(size, M * pow2(-kFarEnd));
  }
  return far;
}

// The rule token by token in fp32, for chunks that the pairs do not hold: n tokens from t0 on, S the
// state's channels 16 t + 4 (lane / 16) + 0..3 of value column col.  Products by chunk would take what
// is not finite to every token of it (0 * NaN in T's and P's zeros); here it reaches later ones only.
template <typename IO, int DK, typename Args>
__device__ __forceinline__ void by_token(const Args &a, f4 *S, int t0, int n, int h, int hk, int col, int lane) {
  constexpr int NT = DK / 16;
  const int g = lane >> 4;
  const IO *kp = static_cast<const IO *>(a.k) + hk * a.Dk + 4 * g, *qp = static_cast<const IO *>(a.q) + hk * a.Dk + 4 * g;
  const IO *vp = static_cast<const IO *>(a.v) + static_cast<long long>(h) * a.Dv + col;
  IO *op = static_cast<IO *>(a.out) + static_cast<long long>(h) * a.Dv + col;
  const bool colin = col < a.Dv;
  typedef typename Vec<IO, 4>::type raw4;
  raw4 kr[NT], qr[NT];   // the next token's, under way
  IO vr = from_f<IO>(0.f);
  float beta_r = 0.f, la_r = 0.f;
  const auto load = [&](int t) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      kr[j] = qr[j] = raw4{};
      if (16 * j + 4 * g < a.Dk) {
        kr[j] = *reinterpret_cast<const raw4 *>(kp + t * a.ks + 16 * j);
        qr[j] = *reinterpret_cast<const raw4 *>(qp + t * a.qs + 16 * j);
      }
    }
    const long long at = static_cast<long long>(t) * a.Hv + h;
    if (colin) vr = vp[t * a.vs];
    beta_r = a.beta[at];
    if (a.log_alpha != nullptr) la_r = a.log_alpha[at];
  };
  load(t0);
#pragma unroll 1
  for (int t = t0; t < t0 + n; ++t) {
    f4 k[NT], q[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        k[j][e] = to_f(static_cast<IO>(kr[j][e]));
        q[j][e] = to_f(static_cast<IO>(qr[j][e]));
      }
    const float v = to_f(vr), beta = beta_r, alpha = __expf(la_r);
    if (t + 1 < t0 + n) load(t + 1);
    const auto dot = [&](const f4 *x, const f4 *y) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fmaf(x[j][e], y[j][e], s);
      return sum_col(s);
    };
    if (a.qk_norm) {
      const float fk = rsqrt_f(dot(k, k) + a.qk_eps), fq = rsqrt_f(dot(q, q) + a.qk_eps);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        k[j] *= fk;
        q[j] *= fq;
      }
    }
    const float d = beta * (v - alpha * dot(S, k)), o = a.scale * fmaf(d, dot(k, q), alpha * dot(S, q));
#pragma unroll
    for (int j = 0; j < NT; ++j) S[j] = d * k[j] + alpha * S[j];
    if (g == 0 && colin) op[t * a.os] = from_f<IO>(o);
  }
}

// A chunk's A operands in the order of their use, kDepth of them under way from LDS: the reads take
// longer than the products that use them, and left to itself the compiler issues them one or two
// ahead.  The order is fixed by keeping the scheduler from moving anything across a step.
// An operand of two parts counts as two.
template <int kDepth, typename At> struct Stream {
  h8 ring[kDepth];
  const At &at;   // at(i): the address of operand i, a compile-time pattern once unrolled
  int total;
  __device__ __forceinline__ Stream(const At &a, int n) : at(a), total(n) {
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
      if (i < n) ring[i] = *reinterpret_cast<const h8 *>(at(i));
    __builtin_amdgcn_sched_barrier(0);
  }
  // operand i, and the next one that has room into its place
  __device__ __forceinline__ h8 take(int i) {
    const h8 x = ring[i % kDepth];
    if (i + kDepth < total) ring[i % kDepth] = *reinterpret_cast<const h8 *>(at(i + kDepth));
    return x;
  }
};

// The kernel's (only) argument, read again where it is used instead of held in registers.
__device__ __forceinline__ auto kernel_args() {
  typedef __attribute__((address_space(4))) const PackedArgs *Args;
  Args a = (Args)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(a));
  return a;
}

template <typename IO, int DK, int MAIN>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2, 2))) void seq_kernel(PackedArgs a) {
  constexpr int NT = DK / 16, NS = DK / 32, NP = kParts<IO>, kCols = 16 * MAIN, kFirstOut = first_out(MAIN);
  using L = Lds<IO, DK, MAIN>;
  using Rec = RecordOf<IO>;
  extern __shared__ __align__(16) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  // the column groups of a head Hv workgroups apart: on one XCD (round robin over 8) if Hv is a
  // multiple of 8, where they share its keys, queries and records in the L2
  const int tile = blockIdx.x / a.Hv, h = blockIdx.x % a.Hv, s = blockIdx.y;
  const int hk = h / (a.Hv / a.Hk);
  const int idx = a.index != nullptr ? a.index[s] : s;
  const bool pooled = a.pool != nullptr;
  if (idx < 0 || (pooled && idx >= a.n_slots)) return;
  if (pooled && a.index != nullptr && __syncthreads_or(seen_before(a, s, idx, tid, 64 * kWaves))) return;
  const bool start = pooled && (a.has == nullptr || a.has[s] != 0);
  int t0, t1;
  seq_range(a, s, t0, t1);
  const int chunks = (t1 - t0 + kC - 1) / kC;
  if (chunks == 0 && (!pooled || start)) return;
  const uint8_t *rec = a.ws + (static_cast<long long>(first_slot(a, s)) * a.Hv + h) * Rec::bytes;
  const long long rec_step = static_cast<long long>(a.Hv) * Rec::bytes;
  const auto left = [&](int c) { return min(kC, t1 - t0 - c * kC); };   // tokens of chunk c
  const auto stage = [&](int c) { return lds + (L::stages == 2 ? (c & 1) * L::stage : 0); };
  const auto hand = [&](int w, int c) { return lds + L::out + (2 * w + (c & 1)) * L::hand; };

  if (wave >= kFirstStaging && wave < kFirstStaging + kStaging) {   // staging: chunk c + 1 while the main waves work on c
    const int hl = tid - 64 * kFirstStaging, cols = min(kCols, a.Dv - tile * kCols);
    const IO *kp = static_cast<const IO *>(a.k) + static_cast<long long>(hk) * a.Dk;
    const IO *vp = static_cast<const IO *>(a.v) + static_cast<long long>(h) * a.Dv + tile * kCols;
    Values<IO, DK, MAIN> values;
    const auto load = [&](Keys<IO, DK> &k, int c) {
      if (c < chunks)
        k.load(Rows<IO>(kp + (t0 + c * kC) * a.ks, left(c), a.ks, a.Dk), static_cast<uint32_t>(a.ks), a.Dk, rec + c * rec_step, hl);
    };
    const auto load_values = [&](int c) {
      if (c < chunks)
        values.load(Rows<IO>(vp + (t0 + c * kC) * a.vs, left(c), a.vs, cols), static_cast<uint32_t>(a.vs), cols,
                    rec + c * rec_step, hl);
    };
    const auto turn = [&](Keys<IO, DK> &k, int c, int ahead) {
      chunk_done<L::stages>(c);
      k.store(stage(c), hl);
      values.store(stage(c), hl);
      load_values(c + 1);
      load(k, c + ahead);
      __syncthreads();
    };
    load_values(0);
    if constexpr (L::stages == 2) {   // keys of two chunks under way, or their loads would be waited for
      Keys<IO, DK> even, odd;
      load(even, 0);
      load(odd, 1);
      for (int c = 0; c < chunks; c += 2) {
        turn(even, c, 2);
        if (c + 1 < chunks) turn(odd, c + 1, 2);
      }
    } else {
      Keys<IO, DK> k;
      load(k, 0);
      for (int c = 0; c < chunks; ++c) turn(k, c, 1);
    }
    __syncthreads();
    return;
  }
  if ((wave >= MAIN && wave < kFirstOut) || wave >= kFirstOut + MAIN) return;

  const int col = tile * kCols + (wave >= kFirstOut ? wave - kFirstOut : wave) * 16 + r;   // this lane's value column
  const bool colin = col < a.Dv;

  if (wave >= kFirstOut) {   // output: chunk c while the main waves work on c + 1
    const int w = wave - kFirstOut;
    const long long slots = a.N / kC + a.n_seqs, q_step = static_cast<long long>(a.Hk) * kQueryBytes<IO, DK>;
    const uint8_t *qp = a.ws + slots * a.Hv * Rec::bytes +
                        (static_cast<long long>(first_slot(a, s)) * a.Hk + hk) * kQueryBytes<IO, DK>;
    IO *op = static_cast<IO *>(a.out) + static_cast<long long>(h) * a.Dv;
    // after the exchange below a lane has row 4 g + r % 4 and four columns from col - r % 4 on
    const uint32_t o_row = static_cast<uint32_t>(a.os) * sizeof(IO);
    const uint32_t o_at = colin ? (4 * g + (r & 3)) * o_row + (col - (r & 3)) * sizeof(IO) : 0x80000000u;   // (no such offset: dropped)
    Output<IO, DK> out;
    const auto finish = [&](int c) {
      f4 x[4], o[4];
      out.query(hand(w, c), lane, x);
      // (a chunk that the main wave has written: dropped)
      const uint32_t o_here = out.values(hand(w, c), lane, x, o) == 0.f ? 0x80000000u : o_at;
      if (c + 1 < chunks) out.load(qp + (c + 1) * q_step, rec + (c + 1) * rec_step, lane);
      const Rows<IO> rows(op + (t0 + c * kC) * a.os, left(c), a.os, a.Dv);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) rows.put4(quad_transpose(o[mt], lane), o_here + 16 * mt * o_row);
    };
    if (chunks > 0) out.load(qp, rec, lane);
    for (int c = 0; c < chunks; ++c) {
      chunk_done<L::stages>(c);
      __syncthreads();
      if (c > 0) finish(c - 1);
    }
    __syncthreads();
    if (chunks > 0) finish(chunks - 1);
    return;
  }

  float *S = pooled ? a.pool + ((static_cast<long long>(idx) * a.Hv + h) * a.Dv + col) * a.Dk : nullptr;
  f4 acc[NT];   // 2^kLift F S^T: channels 16 t + 4 g + 0..3 of column col
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    acc[t] = f4{0.f, 0.f, 0.f, 0.f};
    if (start && colin && 16 * t + 4 * g < a.Dk) {
      float x[4];
      load_n<4>(S + 16 * t + 4 * g, x);
      acc[t] = f4{x[0], x[1], x[2], x[3]} * pow2(kLift);
    }
  }
  int lf = 0;   // F = 2^lf
  const float one = opaque(1.f);
  constexpr std::integral_constant<int, NP> parts{};
  constexpr std::integral_constant<int, 2> two{};
  constexpr std::integral_constant<int, 4> four{};

  int c = 0;
  bool checked = false;   // chunk c is known to hold in the pairs
  while (true) {
    float s0, M;
    bool bad = false;   // what is not finite
    for (; c < chunks; ++c) {
      if (!checked) {
        chunk_done<L::stages>(c);
        __syncthreads();   // stage c is filled
      }
      const uint8_t *st = stage(c);
      uint8_t *ho = hand(wave, c);
      const auto rows = [&](int at, int mt) { return *reinterpret_cast<const f4 *>(st + L::rec + at + 4 * (16 * mt + 4 * g)); };
      // k^ and k^T by K block and row tile, T between them; parts next to each other
      constexpr int nK = 4 * NS * NP, nT = 2 * kFrags, nKT = 2 * NT * NP;
      constexpr int iT = nK, iKT = iT + nT;
      const auto at = [&](int i) -> const uint8_t * {
        if (i < iT) return st + L::K + (i % NP) * L::part + swz<DK * 2>(16 * (i / NP % 4) + r, 4 * (i / NP / 4) + g);
        if (i < iKT) return st + L::rec + Rec::T + (i - iT) % 2 * kFragBytes + ((i - iT) / 2 * 64 + lane) * 16;
        return st + L::KT + ((i - iKT) % NP) * L::part + swz<128>(16 * ((i - iKT) / NP % NT) + r, 4 * ((i - iKT) / NP / NT) + g);
      };
      f4 v[4];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
        v[mt] = *reinterpret_cast<const f4 *>(st + L::V + ((16 * wave + r) * L::v_col + 16 * mt + 4 * g) * 4);
      Stream<kDepth, decltype(at)> ops(at, iKT + nKT);
      // operands i, i + parts, .. times a pair, each onto its own accumulator (fresh: onto zeros),
      // without the products of low parts
      const auto pairs = [&](auto parts, auto n, int i, h8 bh, h8 bl, f4 *c, bool fresh, auto &&beside) {
        constexpr int NPP = decltype(parts)::value, N = decltype(n)::value;
        h8 ah[N], al[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          ah[j] = ops.take(i + j * NPP);
          if constexpr (NPP == 2) al[j] = ops.take(i + j * NPP + 1);
        }
        const f4 zero = {0.f, 0.f, 0.f, 0.f};
        if constexpr (NPP == 2) {
#pragma unroll
          for (int j = 0; j < N; ++j) c[j] = mma(al[j], bh, fresh ? zero : c[j]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) c[j] = mma(ah[j], bl, fresh && NPP == 1 ? zero : c[j]);
#pragma unroll
        for (int j = 0; j < N; ++j) c[j] = mma(ah[j], bh, c[j]);
        beside();   // other work, three instructions between two products
#pragma unroll
        for (int j = 0; j < N * (NPP + 1); ++j) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      const auto give = [&](int at, int k, h8 hi, h8 lo) {   // to the output wave
        *reinterpret_cast<h8 *>(ho + at + (k * L::NE * 64 + lane) * 16) = hi;
        if constexpr (L::NE == 2) *reinterpret_cast<h8 *>(ho + at + ((2 * k + 1) * 64 + lane) * 16) = lo;
      };

      // the column's scale: the largest of its state and of bv V to [2^kTop, 2^(kTop + 1)).  The
      // accumulators stay under the last chunk's scale, f behind, until they are updated.
      float mv = 0.f, ms = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) mv = max4(mv, v[t]);
#pragma unroll
      for (int t = 0; t < NT; ++t) ms = max4(ms, acc[t]);
      mv = max_col(mv);
      ms = max_col(ms);
      // a value, or by its mark in bv a key, gain or decay, that is not finite (a state that is not has no
      // token before it, and stays in its column)
      const bool odd = !(mv < kInf);
      float f;
      int last, below;   // below: the state's exponent below the column's
      {
        const int es = log2_floor(ms), own = es == kNone ? kNone : es - kLift - lf, top = max(log2_floor(mv), own);
        below = top - own;
        int to = top == kNone ? lf : min(kMaxScale, max(-kMaxScale, kTop - top));
        to = min(lf + 126, max(lf - 126, to));
        f = pow2(to - lf);
        last = lf;
        lf = to;
      }

      // X = bv V + bk (k^ S^T)
      f4 x[4];
      h8 bh[NS], bl[NS];
      const float down_s = f * pow2(-kLift);
      const auto split_state = [&](int k) {
        split8(acc[2 * k] * down_s, acc[2 * k + 1] * down_s, one, bh[k], bl[k]);
        give(0, k, bh[k], bl[k]);
      };
      split_state(0);
      __builtin_amdgcn_sched_barrier(0);
      f4 rbk[4], rdt[4], rdc[4];   // row factors, read while the first products run
      float ec = 0.f;
      int held = 0;
      bool ask = false;
#pragma unroll
      for (int k = 0; k < NS; ++k)
        pairs(parts, four, k * 4 * NP, bh[k], bl[k], x, k == 0, [&] {
          if (k == 0) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) rbk[mt] = rows(Rec::bk, mt);
            const float2 e = *reinterpret_cast<const float2 *>(st + L::rec + Rec::ec);
            ec = e.x * f;
            held = __float_as_int(e.y);
          }
          if (k + 1 < NS) split_state(k + 1);
          // (most chunks under weak decays are held up by each column's state alone)
          if (k + 1 == NS) ask = odd || below > held;
        });
      // not for the pairs?  (Asked here, where the answer is there without a wait; the state is as it was.)
      if (__builtin_expect(__any(ask), false) && !checked) {
        s0 = ms * pow2(-kLift - last);
        M = __builtin_elementwise_maximum(mv, s0);
        const f4 words = *reinterpret_cast<const f4 *>(st + L::rec + Rec::ec);
        const float decay = words[0], d1 = words[2], d3 = d1 * d1 * d1;   // (no three tokens decay by more than d3)
        // Is a size far below M out of the question?  Every four rows have one that carries the next four, or
        // every row holds its own, or the one before holds it up.  (Comparisons that NaN passes.)
        float low = kInf, each = kInf, end = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          low = fminf(low, max4(0.f, v[t]));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            end = e == 0 ? fabsf(v[t][0]) : fmaxf(fabsf(v[t][e]), fabsf(v[t][e - 1]) * d1);
            each = fminf(each, end);
          }
        }
        low = g == 0 ? fminf(low, fmaxf(fabsf(v[0][0]), s0)) : low;
        each = g == 3 ? fminf(each, end * pow2(kFarEnd - kFarBefore<IO>)) : each;
        bad = __any(odd);
        if (bad || (__any(low * (d3 * d3 * d1) < M * pow2(-kNear<IO>)) && __any(each < M * pow2(-kFarBefore<IO>)))) {
          int here = lane;
          asm volatile("" : "+v"(here));
          const float *column = reinterpret_cast<const float *>(st + L::V) + (16 * wave + (here & 15)) * L::v_col;
          const bool near = clearly_near<IO>(column, s0, M, decay, d3, left(c), here >> 4);
          if (bad || __any(!near)) {
            lf = last;
            break;
          }
        }
      }
      checked = false;
      {
        const float F = pow2(lf);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) x[mt] = rbk[mt] * x[mt] + v[mt] * F;
      }
      // E = T X, in halves of 32 rows: X's second half is split beside the products of the first, the
      // state's decay and E's first half follow beside them
      f4 d[4], ed[4];
      float mx = 0.f, me = 0.f;   // largest of a column's X and E, of this lane's rows
      h8 xh[2], xl[2], eh[2], el[2];
      const auto split_x = [&](int k) { split8(x[2 * k], x[2 * k + 1], one, xh[k], xl[k]); };
      const auto finish_e = [&](int k) {   // E's rows 32 k ..: as they are, and as the update takes them
#pragma unroll
        for (int mt = 2 * k; mt < 2 * k + 2; ++mt) {
          ed[mt] = rdt[mt] * d[mt];
          me = max4(me, ed[mt]);
        }
      };
      const auto split_e = [&](int k) { split8(rdc[2 * k] * d[2 * k], rdc[2 * k + 1] * d[2 * k + 1], one, eh[k], el[k]); };
      const auto give_e = [&](int k) {
        h8 oh, ol;
        split8(ed[2 * k], ed[2 * k + 1], one, oh, ol);
        give(L::E, k, oh, ol);
      };
      split_x(0);
      __builtin_amdgcn_sched_barrier(0);
      pairs(two, four, iT, xh[0], xl[0], d, true, [&] {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          rdt[mt] = rows(Rec::dt, mt);
          rdc[mt] = rows(Rec::dc, mt);
        }
        split_x(1);
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] *= ec;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) mx = max4(mx, x[mt]);
      });
      pairs(two, two, iT + 2 * 4, xh[1], xl[1], d + 2, false, [&] {
        finish_e(0);
        split_e(0);
      });
      finish_e(1);
      float down = 1.f;
      if (__builtin_expect(__any(mx > kOver || me > kOver), false)) {
        // past fp16's range: the columns are brought down, and E formed again
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {   // (where X did not fit, E says nothing yet)
          mx = max_col(mx);
          const int over = log2_floor(mx <= kOver ? max_col(me) : mx);
          const int to = over == kNone ? lf : max(-kMaxScale, min(lf, lf + kTop - over));
          const float now = pow2(to - lf);
          lf = to;
          down *= now;
          mx = me = 0.f;
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[t] *= now;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            x[mt] *= now;
            mx = max4(mx, x[mt]);
          }
          split_x(0);
          split_x(1);
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            d[mt] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k <= mt / 2; ++k) {
              const uint8_t *p = at(iT + 2 * frag_of(mt, k));
              const h8 th = *reinterpret_cast<const h8 *>(p), tl = *reinterpret_cast<const h8 *>(p + kFragBytes);
              d[mt] = mma(tl, xh[k], d[mt]);
              d[mt] = mma(th, xl[k], d[mt]);
              d[mt] = mma(th, xh[k], d[mt]);
            }
          }
          finish_e(0);
          finish_e(1);
          if (!__any(mx > kOver || me > kOver)) break;
        }
        split_e(0);
      }
      // S <- e^{g_C} S + (e^{g_C - g} E)^T k^; beside the products E's second half, then its parts for
      // the output wave
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int t = 0; t < NT; t += 4)
          pairs(parts, four, iKT + (k * NT + t) * NP, eh[k], el[k], acc + t, false, [&] {
            if (k == 0 && t == 0) split_e(1);
            if (t + 4 == NT) give_e(k);
          });
      if (g == 0) {
        float *scale = reinterpret_cast<float *>(ho + L::scale) + r;
        scale[0] = down;
        scale[16] = pow2(-lf);
      }
    }
    if (c >= chunks) break;
    // (what the other path needs is formed here, not kept over the loop)
    int here = lane;
    asm volatile("" : "+v"(here));
    if (!bad) {
      const float *column = reinterpret_cast<const float *>(stage(c) + L::V) + (16 * wave + (here & 15)) * L::v_col;
      checked = !__any(falls_far<IO>(*kernel_args(), column, s0, M, t0 + c * kC, left(c), h, here));
      if (checked) continue;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] *= pow2(-kLift - lf);
    by_token<IO, DK>(*kernel_args(), acc, t0 + c * kC, left(c), h, hk, col, here);
    lf = -kLift;
    if (here < 16) reinterpret_cast<float *>(hand(wave, c) + L::scale)[16 + here] = 0.f;
    ++c;
  }
  __syncthreads();
  if (pooled && colin) {
    const float f = pow2(-kLift - lf);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float x[4] = {acc[t][0] * f, acc[t][1] * f, acc[t][2] * f, acc[t][3] * f};
      if (16 * t + 4 * g < a.Dk) store_n<4>(S + 16 * t + 4 * g, x);
    }
  }
}

template <typename IO, int DK, int MAIN>
hipError_t launch_seq(const PackedArgs &a, hipStream_t s) {
  const auto kernel = seq_kernel<IO, DK, MAIN>;
  using L = Lds<IO, DK, MAIN>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, L::bytes);
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<unsigned>((a.Dv + L::cols - 1) / L::cols) * a.Hv, a.n_seqs);
  hipLaunchKernelGGL(kernel, grid, dim3(64 * kWaves), L::bytes, s, a);
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_io(const PackedArgs &a, hipStream_t s) {
  const long long slots = a.N / kC + a.n_seqs;
  const dim3 grid(static_cast<unsigned>(slots * a.Hv));
  if (a.Dk > 64)
    hipLaunchKernelGGL((prep_kernel<IO, 128>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((prep_kernel<IO, 64>), grid, dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if ((a.Dv + 15) / 16 * static_cast<long long>(a.Hv) * a.n_seqs <= kCus)
    return a.Dk > 64 ? launch_seq<IO, 128, 1>(a, s) : launch_seq<IO, 64, 1>(a, s);
  return a.Dk > 64 ? launch_seq<IO, 128, 2>(a, s) : launch_seq<IO, 64, 2>(a, s);
}

}  // namespace

// Keys up to 64 channels run as 64, others as 128, filled up with zeros; both sides are read eight
// channels at a time.  (Token by token, the other kernel takes 65 ms for 32768 tokens against 1.1, 7.6 ms
// for 4 x 4096 against 0.2, and 325 us for 23 short sequences against 41.)
bool packed_chunk_supports(const gdr_packed_desc_t &d) { return d.Dk % 8 == 0 && d.Dv % 8 == 0; }

uint64_t packed_chunk_ws_bytes(const gdr_packed_desc_t &d) {
  const uint64_t slots = static_cast<uint64_t>(d.n_tokens) / kC + d.n_seqs;
  const uint64_t rec = d.io_dtype == GDR_BF16 ? RecordOf<uint16_t>::bytes : RecordOf<float>::bytes;
  const uint64_t q = d.io_dtype == GDR_F32 ? kQueryBytes<float, 64> : kQueryBytes<uint16_t, 64>;
  return slots * (d.Hv * rec + d.Hk * q * (d.Dk > 64 ? 2 : 1));
}

hipError_t launch_packed_chunk(const PackedArgs &a, int io_dtype, hipStream_t s) {
  return io_dtype == GDR_BF16 ? launch_io<uint16_t>(a, s)
         : io_dtype == GDR_F16 ? launch_io<_Float16>(a, s) : launch_io<float>(a, s);
}

}  // namespace gdr
