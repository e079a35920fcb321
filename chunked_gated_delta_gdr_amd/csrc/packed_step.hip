// The gated delta rule token by token over a pool of states: gdr_packed_step, and gdr_packed_fwd
// for the shapes the chunked kernel does not take.
//
// Per sequence, value head and token
//     S <- alpha S;  d = beta (v - S k);  S <- S + d k^T;  o = scale S q
// Every state row r is independent given k and q, with the old state
//     x = S_r . k,  y = S_r . q,  d = beta (v_r - alpha x),  o_r = scale (alpha y + d (k . q)),
//     S_r <- alpha S_r + d k
// so a token needs one look at the state.  A workgroup holds 128 rows of one (sequence, head) in
// registers (16 lanes a row, 8 rows a lane at most) for all of the sequence's tokens and touches
// the pool once at each end: bound by HBM, 8 Dv Dk bytes a (sequence, head).
// Measured: 64 sequences x 32 heads of 128 x 128, one token each, 270 MB: 43 us in a loop over one pool
// (6.3 TB/s, half of the reads from the last-level cache), 61 over four pools in turn (4.4 TB/s); one
// sequence 7.1 us (latency: a load of the token, the state and one row sum after another); 96 sequences
// x 12 heads of 64 x 96 with 1 to 4 tokens 16 us, bound by its instructions a token.  8 rows a lane: the state of a workgroup is 64 KB of registers, three
// workgroups a CU under way (five of half the size with 64 columns).
// The output norm needs all Dv rows of a head: it is fused up to 256, with twice the threads from 129 on
// (as a pass of its own it would read a rounded o: 1.4 times the error of one rounding).
#include <utility>

#include "packed.h"

namespace gdr {
namespace {

constexpr int kThreads = 256, kWide = 512;
constexpr int rows_of(int threads) { return threads / 2; }   // state rows of a workgroup
constexpr int kRpl = 8;      // rows of a lane, at most

// What one token brings, as loaded: kept raw until its turn, so that nothing waits for it before.
template <typename IO, int NC> struct Token {
  IO k[NC], q[NC], v;   // v: lane p of a row group has the group's p-th row
  float beta, la;
};

// lane p's value to its 16 lanes
template <int P> __device__ __forceinline__ float from_lane(float x) { return dpp<0x150 + P>(x); }
template <int... P> __device__ __forceinline__ void spread(float x, float *out, std::integer_sequence<int, P...>) {
  ((out[P] = from_lane<P>(x)), ...);
}

// DK: 128 or 64 (the pool 16-byte aligned: columns in runs of four, 16-byte loads), or 0: any Dk <= 128
// and alignment, an element a load.
// kMulti: the sequences' lengths come from cu_seqlens (else one token each).
template <typename IO, int DK, bool kMulti, int THREADS>
__global__ __launch_bounds__(THREADS, THREADS == kWide ? 2 : DK == 64 ? 5 : 3) void recur_kernel(PackedArgs a) {
  constexpr int kRows = rows_of(THREADS);
  constexpr int NC = DK == 64 ? 4 : 8;   // columns of a lane
  __shared__ float red[2][THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 15, grp = tid >> 4;
  const int s = blockIdx.y, h = blockIdx.x % a.Hv, r0 = (blockIdx.x / a.Hv) * kRows;
  const int hk = h / (a.Hv / a.Hk);
  const int nrows = min(kRows, a.Dv - r0);
  const int rpl = (nrows + THREADS / 16 - 1) / (THREADS / 16);   // rows of a lane here
  const int row0 = grp * rpl;
  const int mine = min(rpl, nrows - row0);        // may be <= 0
  const auto col = [&](int j) { return DK != 0 ? (j >> 2) * 64 + lane * 4 + (j & 3) : lane + 16 * j; };

  int t0, t1;
  seq_range(a, s, t0, t1);
  const int idx = a.index != nullptr ? a.index[s] : s;
  const bool pooled = a.pool != nullptr;
  const bool start = pooled && (a.has == nullptr || a.has[s] != 0);
  // (the first token does not wait for the slot)
  const IO *q = static_cast<const IO *>(a.q) + hk * a.Dk;
  const IO *k = static_cast<const IO *>(a.k) + hk * a.Dk;
  const IO *v = static_cast<const IO *>(a.v) + h * a.Dv + r0 + row0 + lane;
  IO *out = static_cast<IO *>(a.out) + h * a.Dv + r0 + row0 + lane;
  const auto load = [&](int t, Token<IO, NC> &x) {
    const long long qo = t * a.qs, ko = t * a.ks;
    if (DK != 0) {
      typedef typename Vec<IO, 4>::type raw4;
#pragma unroll
      for (int f = 0; f < NC / 4; ++f) {
        const raw4 kr = *reinterpret_cast<const raw4 *>(k + ko + f * 64 + lane * 4);
        const raw4 qr = *reinterpret_cast<const raw4 *>(q + qo + f * 64 + lane * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x.k[4 * f + e] = kr[e];
          x.q[4 * f + e] = qr[e];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const bool in = col(j) < a.Dk;
        x.k[j] = in ? k[ko + col(j)] : from_f<IO>(0.f);
        x.q[j] = in ? q[qo + col(j)] : from_f<IO>(0.f);
      }
    }
    x.v = lane < mine ? v[t * a.vs] : from_f<IO>(0.f);
    const long long g = static_cast<long long>(t) * a.Hv + h;
    x.beta = a.beta[g];
    x.la = a.log_alpha != nullptr ? a.log_alpha[g] : 0.f;
  };
  Token<IO, NC> cur;
  if (t0 < t1) load(t0, cur);

  // (without a pool a slot is only a sequence's mark: negative skips it)
  if (idx < 0 || (pooled && idx >= a.n_slots)) return;
  float *S = pooled ? a.pool + ((static_cast<long long>(idx) * a.Hv + h) * a.Dv + r0) * a.Dk : nullptr;

  float st[kRpl][NC];
#pragma unroll
  for (int p = 0; p < kRpl; ++p) {
    const bool in = start && p < mine;
    if (DK != 0) {
#pragma unroll
      for (int f = 0; f < NC / 4; ++f) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in) x = *reinterpret_cast<const float4 *>(S + static_cast<long long>(row0 + p) * DK + f * 64 + lane * 4);
        st[p][4 * f] = x.x; st[p][4 * f + 1] = x.y; st[p][4 * f + 2] = x.z; st[p][4 * f + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < NC; ++j)
        st[p][j] = in && col(j) < a.Dk ? S[static_cast<long long>(row0 + p) * a.Dk + col(j)] : 0.f;
    }
  }

  // a slot that an earlier sequence names is that one's
  if (pooled && a.index != nullptr && __syncthreads_or(seen_before(a, s, idx, tid, THREADS))) return;

  const bool norm = a.norm_w != nullptr && a.Dv <= kRows;
#pragma unroll 1
  for (int t = t0; t < t1; ++t) {
    Token<IO, NC> nxt;
    if (kMulti && t + 1 < t1) load(t + 1, nxt);
    float kt[NC], qt[NC], vt[kRpl], kq = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      kt[j] = to_f(cur.k[j]);
      qt[j] = to_f(cur.q[j]);
    }
    spread(to_f(cur.v), vt, std::make_integer_sequence<int, kRpl>());
    if (a.qk_norm) {
      float kk = 0.f, qq = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        kk = fmaf(kt[j], kt[j], kk);
        qq = fmaf(qt[j], qt[j], qq);
      }
      kk = rsqrt_f(sum16(kk) + a.qk_eps);
      qq = rsqrt_f(sum16(qq) + a.qk_eps);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        kt[j] *= kk;
        qt[j] *= qq;
      }
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) kq = fmaf(kt[j], qt[j], kq);
    kq = sum16(kq);
    // (off by 2^-24 |la| of itself: nothing where it matters, near 1)
    const float alpha = a.log_alpha != nullptr ? __expf(cur.la) : 1.f;
    float o[kRpl];
#pragma unroll
    for (int p = 0; p < kRpl; ++p) {
      o[p] = 0.f;
      if (p >= rpl) continue;   // (alike in the workgroup)
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        x = fmaf(st[p][j], kt[j], x);
        y = fmaf(st[p][j], qt[j], y);
      }
      x = sum16(x);
      y = sum16(y);
      const float d = cur.beta * (vt[p] - alpha * x);
      o[p] = a.scale * fmaf(d, kq, alpha * y);
#pragma unroll
      for (int j = 0; j < NC; ++j) st[p][j] = fmaf(d, kt[j], alpha * st[p][j]);
    }
    // lane p of a row group stores its p-th row
    float ov = 0.f;
#pragma unroll
    for (int p = 0; p < kRpl; ++p) ov = lane == p ? o[p] : ov;
    if (norm) {
      const float ss = sum_lanes<64>(lane < mine ? ov * ov : 0.f);
      if ((tid & 63) == 0) red[t & 1][tid >> 6] = ss;
      __syncthreads();
      float all = red[t & 1][0];
#pragma unroll
      for (int w = 1; w < THREADS / 64; ++w) all += red[t & 1][w];
      const float r = rsqrt_f(all / a.Dv + a.norm_eps);
      if (lane < mine) {
        ov *= r * to_f(static_cast<const IO *>(a.norm_w)[row0 + lane]);
        if (a.norm_z != nullptr) ov *= silu_f<IO>(to_f(static_cast<const IO *>(a.norm_z)[t * a.zs + h * a.Dv + row0 + lane]));
      }
    }
    if (lane < mine) out[t * a.os] = from_f<IO>(ov);
    if (kMulti) cur = nxt;
  }

  if (!pooled || (t0 == t1 && start)) return;
#pragma unroll
  for (int p = 0; p < kRpl; ++p) {
    if (p >= mine) continue;
    if (DK != 0) {
#pragma unroll
      for (int f = 0; f < NC / 4; ++f)
        *reinterpret_cast<float4 *>(S + static_cast<long long>(row0 + p) * DK + f * 64 + lane * 4) =
            make_float4(st[p][4 * f], st[p][4 * f + 1], st[p][4 * f + 2], st[p][4 * f + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < NC; ++j)
        if (col(j) < a.Dk) S[static_cast<long long>(row0 + p) * a.Dk + col(j)] = st[p][j];
    }
  }
}

template <typename IO, int DK, int THREADS>
hipError_t launch_rows(const PackedArgs &a, hipStream_t s) {
  constexpr int rows = rows_of(THREADS);
  const dim3 grid(static_cast<unsigned>(a.Hv) * ((a.Dv + rows - 1) / rows), a.n_seqs);
  if (a.cu != nullptr)
    hipLaunchKernelGGL((recur_kernel<IO, DK, true, THREADS>), grid, dim3(THREADS), 0, s, a);
  else
    hipLaunchKernelGGL((recur_kernel<IO, DK, false, THREADS>), grid, dim3(THREADS), 0, s, a);
  return hipGetLastError();
}

template <typename IO, int DK>
hipError_t launch_dk(const PackedArgs &a, hipStream_t s) {
  if (a.norm_w != nullptr && a.Dv > rows_of(kThreads) && a.Dv <= rows_of(kWide)) return launch_rows<IO, DK, kWide>(a, s);
  return launch_rows<IO, DK, kThreads>(a, s);
}

template <typename IO>
hipError_t launch_io(const PackedArgs &a, hipStream_t s) {
  const bool aligned = (reinterpret_cast<uintptr_t>(a.pool) & 15u) == 0;
  if (aligned && a.Dk == 128) return launch_dk<IO, 128>(a, s);
  if (aligned && a.Dk == 64) return launch_dk<IO, 64>(a, s);
  return launch_dk<IO, 0>(a, s);
}

// The output norm as a pass of its own, in place: for the chunked kernel, whose workgroups hold 32 of a
// row's columns, and for Dv > 256.  A row is (token, head), 64 lanes a row, Dv <= 512; it reads and
// writes what the kernel before left in the caches.  So o is rounded to the io type before its norm as well,
// 1.4 times the error of one rounding: kept in fp32 it would need a workspace of another 4 Dv bytes a token
// and head, which the workspace's size, a matter of the descriptor alone, would ask of every call.
template <typename IO>
__device__ __forceinline__ void norm_row(const PackedArgs &a, int t, int h, int lane) {
  int s = t;
  if (a.cu != nullptr) {   // the last sequence that begins at or before t
    int lo = 0, hi = a.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (clamp_tok(a.cu[mid], a.N) <= t) lo = mid; else hi = mid;
    }
    s = lo;
    int t0, t1;
    seq_range(a, s, t0, t1);
    if (t < t0 || t >= t1) return;
  }
  if (a.index != nullptr) {
    const int idx = a.index[s];
    if (idx < 0 || (a.pool != nullptr && idx >= a.n_slots)) return;
    if (a.pool != nullptr && __any(seen_before(a, s, idx, lane, 64))) return;
  }
  IO *o = static_cast<IO *>(a.out) + t * a.os + static_cast<long long>(h) * a.Dv;
  float x[8], ss = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = lane + 64 * j < a.Dv ? to_f(o[lane + 64 * j]) : 0.f;
    ss = fmaf(x[j], x[j], ss);
  }
  const float r = rsqrt_f(sum_lanes<64>(ss) / a.Dv + a.norm_eps);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = lane + 64 * j;
    if (c >= a.Dv) continue;
    float y = x[j] * r * to_f(static_cast<const IO *>(a.norm_w)[c]);
    if (a.norm_z != nullptr) y *= silu_f<IO>(to_f(static_cast<const IO *>(a.norm_z)[t * a.zs + static_cast<long long>(h) * a.Dv + c]));
    o[c] = from_f<IO>(y);
  }
}

// Workgroups of a launch, at most: its work-items have to stay below 2^32
constexpr long long kNormGroups = 1ll << 23;
template <typename IO>
__global__ __launch_bounds__(256) void packed_norm_kernel(PackedArgs a) {
  const long long rows = static_cast<long long>(a.N) * a.Hv;
  for (long long row = blockIdx.x * 4ll + (threadIdx.x >> 6); row < rows; row += gridDim.x * 4ll)
    norm_row<IO>(a, static_cast<int>(row / a.Hv), static_cast<int>(row % a.Hv), threadIdx.x & 63);
}

}  // namespace

hipError_t launch_packed_recur(const PackedArgs &a, int io_dtype, hipStream_t s) {
  hipError_t e = io_dtype == GDR_BF16 ? launch_io<uint16_t>(a, s)
                 : io_dtype == GDR_F16 ? launch_io<_Float16>(a, s) : launch_io<float>(a, s);
  if (e == hipSuccess && a.norm_w != nullptr && a.Dv > rows_of(kWide)) e = launch_packed_norm(a, io_dtype, s);
  return e;
}

hipError_t launch_packed_norm(const PackedArgs &a, int io_dtype, hipStream_t s) {
  const long long rows = static_cast<long long>(a.N) * a.Hv;
  if (rows == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(rows < 4 * kNormGroups ? (rows + 3) / 4 : kNormGroups)), block(256);
  if (io_dtype == GDR_BF16)
    hipLaunchKernelGGL((packed_norm_kernel<uint16_t>), grid, block, 0, s, a);
  else if (io_dtype == GDR_F16)
    hipLaunchKernelGGL((packed_norm_kernel<_Float16>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((packed_norm_kernel<float>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace gdr
