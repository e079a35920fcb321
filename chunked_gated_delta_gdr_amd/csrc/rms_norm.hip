// Root-mean-square norm of rows, with the residual's addition in front, a SiLU gate behind, an
// output in io type or in 8 bits with a scale per row, and its gradient.
//
//     h = x + res,  r = 1 / sqrt(mean(h^2) + eps),  n = h r,  y = n (.) w (.) silu(z)
//     8 bits: s = max|y| / 127 (int8) or / 448 (e4m3), code = round(y / s)
//     u = dy (.) w (.) silu(z),  dx = r (u - n mean(u (.) n)) + d_res,
//     dw = sum over rows of dy (.) silu(z) (.) n,  dz = dy (.) w (.) n (.) silu'(z)
//
// Bound by HBM: a row is read once into registers (8 to 1024 lanes a row, 16 bytes a lane
// and load), every statistic is a reduction over those lanes in fp32, and the outputs are written
// from the registers.  Row starts need no alignment beyond the element's.
//
// Measured (bf16): 16384 x 4096 with residual into e4m3 90 us, 470 MB (5.2 TB/s); 262144 x 128 gated 37 us
// (5.4 TB/s); 8 rows of 4096 4.8 us, where the call from Python takes 8.7.  Over 64 to 16384 channels
// 33 M elements run at 6.0 to 6.6 TB/s where the lanes are filled and rows start on 16 bytes, 4.7 to 6 elsewhere
// (the last-level cache holds a part).  Gradient: 8191 x 2048 24 us, and 65537 x 128 gated (fp16) 18 us,
// 5 and 4 more for the weight's sum; 2.7 to 3.5 TB/s at widths that leave lanes idle or whose rows end inside a
// load (300, 700, 1300, 2304, 5000, 7001, 12000 channels), against 5 to 5.5 at 1024, 2048 and 4096.
#include <type_traits>

#include "packed.h"

namespace gdr {
namespace {

// threads of a workgroup: a row's lanes where they are more than a wave, else four waves
constexpr int threads_of(int lanes) { return lanes > 64 ? lanes : 256; }

template <typename IO> constexpr int kVec = 16 / static_cast<int>(sizeof(IO));   // elements of a load

// elements c .. c + V - 1 of a row of D: zeros past its end
template <int V, typename IO> __device__ __forceinline__ void load_row(const IO *p, int c, int D, float *x) {
  if (c + V <= D) {
    load_n<V>(p + c, x);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = c + e < D ? to_f(p[c + e]) : 0.f;
  }
}
// the same as they are stored
template <int V, typename IO> using Raw = typename Vec<IO, V>::type;
template <int V, typename IO> __device__ __forceinline__ Raw<V, IO> load_raw(const IO *p, int c, int D) {
  if (c + V <= D) return *reinterpret_cast<const Raw<V, IO> *>(p + c);
  Raw<V, IO> x;
#pragma unroll
  for (int e = 0; e < V; ++e) x[e] = c + e < D ? p[c + e] : IO(0);
  return x;
}
template <int V, typename IO> __device__ __forceinline__ void store_row(IO *p, int c, int D, const float *x) {
  if (c + V <= D) {
    store_n<V>(p + c, x);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c + e < D) p[c + e] = from_f<IO>(x[e]);
  }
}

// sum (or NaN-keeping max) over a row's lanes; over the waves of a wider row through red
template <int LANES> __device__ __forceinline__ float row_sum(float x, float *red) {
  x = sum_lanes<(LANES > 64 ? 64 : LANES)>(x);
  if (LANES > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < LANES / 64; ++i) x += red[i];
  }
  return x;
}
template <int LANES> __device__ __forceinline__ void row_sum2(float &x, float &y, float (*red)[16]) {
  x = sum_lanes<(LANES > 64 ? 64 : LANES)>(x);
  y = sum_lanes<(LANES > 64 ? 64 : LANES)>(y);
  if (LANES > 64) {
    if ((threadIdx.x & 63) == 0) {
      red[0][threadIdx.x >> 6] = x;
      red[1][threadIdx.x >> 6] = y;
    }
    __syncthreads();
    x = red[0][0];
    y = red[1][0];
#pragma unroll
    for (int i = 1; i < LANES / 64; ++i) {
      x += red[0][i];
      y += red[1][i];
    }
  }
}
template <int LANES> __device__ __forceinline__ float row_max(float x, float *red) {
  x = max_lanes<(LANES > 64 ? 64 : LANES)>(x);
  if (LANES > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < LANES / 64; ++i) x = max_nan(x, red[i]);
  }
  return x;
}

// four codes in a word; values are within the type's range but for rounding
__device__ __forceinline__ uint32_t pack_int8(const float *y) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int q = static_cast<int>(rintf(y[e]));   // (NaN: 0)
    w |= (static_cast<uint32_t>(min(127, max(-127, q))) & 0xffu) << (8 * e);
  }
  return w;
}
__device__ __forceinline__ uint32_t pack_fp8(const float *y) {
  float c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = y[e] > 448.f ? 448.f : (y[e] < -448.f ? -448.f : y[e]);   // (keeps NaN)
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
  return static_cast<uint32_t>(w);
}

template <typename IO, int LANES, int IT>
__global__ __launch_bounds__(threads_of(LANES)) void norm_kernel(NormArgs a) {
  constexpr int V = kVec<IO>, R = threads_of(LANES) / LANES;
  __shared__ float red[2][16];
  const int l = threadIdx.x % LANES;
  const long long row = static_cast<long long>(blockIdx.x) * R + threadIdx.x / LANES;
  const bool live = row < a.rows;   // (with 256 lanes a row and more every workgroup has one)
  const int D = live ? a.D : 0;     // a dead row loads and stores nothing
  const IO *x = static_cast<const IO *>(a.x) + (live ? row * a.xs : 0);
  const IO *res = a.res != nullptr ? static_cast<const IO *>(a.res) + (live ? row * a.rs : 0) : nullptr;
  const IO *z = a.z != nullptr ? static_cast<const IO *>(a.z) + (live ? row * a.zs : 0) : nullptr;
  float h[IT][V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < IT; ++i) load_row<V>(x, (i * LANES + l) * V, D, h[i]);
  if (res != nullptr) {
    float b[IT][V];
#pragma unroll
    for (int i = 0; i < IT; ++i) load_row<V>(res, (i * LANES + l) * V, D, b[i]);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) h[i][e] += b[i][e];
      store_row<V>(static_cast<IO *>(a.res_out) + row * a.D, (i * LANES + l) * V, D, h[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) ss = fmaf(h[i][e], h[i][e], ss);
  const float r = rsqrt_f(row_sum<LANES>(ss, red[0]) * a.inv_d + a.eps);
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (i * LANES + l) * V;
    float g[V];
#pragma unroll
    for (int e = 0; e < V; ++e) h[i][e] *= r;
    if (a.w != nullptr) {
      load_row<V>(static_cast<const IO *>(a.w), c, D, g);
#pragma unroll
      for (int e = 0; e < V; ++e) h[i][e] *= g[e];
    }
    if (z != nullptr) {
      load_row<V>(z, c, D, g);
#pragma unroll
      for (int e = 0; e < V; ++e) h[i][e] *= silu_f<IO>(g[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) m = c + e < D ? max_nan(m, fabsf(h[i][e])) : m;
  }
  if (a.out_kind == GDR_OUT_IO) {
#pragma unroll
    for (int i = 0; i < IT; ++i) store_row<V>(static_cast<IO *>(a.y) + row * a.D, (i * LANES + l) * V, D, h[i]);
    return;
  }
  const bool fp8 = a.out_kind == GDR_OUT_FP8;
  float scale = row_max<LANES>(m, red[1]) / (fp8 ? 448.f : 127.f);
  if (scale < 1.17549435e-38f) scale = 0.f;   // a row of zeros (or one whose reciprocal scale would overflow)
  const float inv = scale == 0.f ? 0.f : 1.f / scale;
  const float step = scale < __int_as_float(0x7f800000) ? scale : 0.f;   // (an infinite one: finite y / s are 0, not 0 * inf)
  if (live && l == 0) a.scales[row] = scale;
  uint8_t *y = static_cast<uint8_t *>(a.y) + row * a.D;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (i * LANES + l) * V;
    uint32_t w[V / 4];
#pragma unroll
    for (int e = 0; e < V; ++e) {   // y / s to the last bit or so: a product, and its rest (16-bit inputs make
                                     // exact ties often, one code in 10^5: these go by y's own fp32 roundings)
      const float c0 = h[i][e] * inv;
      h[i][e] = fmaf(fmaf(-c0, step, h[i][e]), inv, c0);
    }
#pragma unroll
    for (int e = 0; e < V; e += 4) w[e / 4] = fp8 ? pack_fp8(h[i] + e) : pack_int8(h[i] + e);
    if (c + V <= D) {
      typedef uint32_t words __attribute__((ext_vector_type(V / 4), aligned(1)));
      words o;
#pragma unroll
      for (int e = 0; e < V / 4; ++e)
        if constexpr (V == 4) o = w[0]; else o[e] = w[e];
      *reinterpret_cast<words *>(y + c) = o;
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e < D) y[c + e] = static_cast<uint8_t>(w[e / 4] >> (8 * (e & 3)));
    }
  }
}

// waves a SIMD that the gradient's registers leave room for without spilling (the compiler is held to
// them: 129 registers instead of 128 would cost a wave)
constexpr int bwd_waves(int lanes, int it, int vec) { return lanes == 1024 || it == 1 ? 4 : it * vec > 16 ? 2 : 3; }

// Gradient.  A workgroup takes every groups-th block of rows, keeps its part of dw in registers
// and leaves it in part[group][D]; dw_kernel adds the parts in their order.
// kGate: with the gate's gradient (its registers would cost the other a workgroup a CU: 8191 x 2048 took
// 41 us in one kernel for both, 36 in two).
template <typename IO, int LANES, int IT, bool kGate>
__global__ __launch_bounds__(threads_of(LANES), bwd_waves(LANES, IT, kVec<IO>)) void norm_bwd_kernel(NormArgs a) {
  constexpr int V = kVec<IO>, R = threads_of(LANES) / LANES;
  // with 16 elements a lane and more the weight and the gate are read a second time, from the caches,
  // instead of held over the row's sums (bf16, 16384 channels, gated: 1.1 TB/s held, which spills,
  // 4.1 read again; 2048 fp32 channels, 8 elements a lane: 6.3 held, 5.9 read again)
  constexpr bool kTwice = IT * V >= 16;
  constexpr int kHeld = kTwice ? 1 : IT;
  __shared__ float red[4][16];
  const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  float dw[IT][V];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[i][e] = 0.f;
  int turn = 0;
  for (long long base = static_cast<long long>(blockIdx.x) * R; base < a.rows;
       base += static_cast<long long>(a.groups) * R, turn ^= 2) {
    const long long row = base + sub;
    const bool live = row < a.rows;
    const int D = live ? a.D : 0;
    const IO *x = static_cast<const IO *>(a.x) + (live ? row * a.xs : 0);
    const IO *dy = static_cast<const IO *>(a.dy) + (live ? row * a.ds : 0);
    const IO *z = kGate ? static_cast<const IO *>(a.z) + (live ? row * a.zs : 0) : nullptr;
    const IO *res = a.res != nullptr ? static_cast<const IO *>(a.res) + (live ? row * a.rs : 0) : nullptr;
    Raw<V, IO> hr[IT], ur[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) hr[i] = load_raw<V>(x, (i * LANES + l) * V, D);
#pragma unroll
    for (int i = 0; i < IT; ++i) ur[i] = load_raw<V>(dy, (i * LANES + l) * V, D);
    float ss = 0.f, uh = 0.f, w[kHeld][V], dz[kHeld][V], u[kHeld][V];
    // block i's u = dy (.) silu(z), its weight, and dz but for n
    auto factors = [&](int i) {
      const int c = (i * LANES + l) * V, j = i % kHeld;
      if (a.w != nullptr) load_row<V>(static_cast<const IO *>(a.w), c, D, w[j]);
      if (kGate) load_row<V>(z, c, D, dz[j]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (a.w == nullptr) w[j][e] = 1.f;
        u[j][e] = to_f(static_cast<IO>(ur[i][e]));
        if (kGate) {
          const float g = dz[j][e], sg = sigmoid_f<IO>(g);
          dz[j][e] = u[j][e] * w[j][e] * sg * (1.f + g * (1.f - sg));
          u[j][e] *= g * sg;
        }
      }
    };
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int j = i % kHeld;
      factors(i);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float h = to_f(static_cast<IO>(hr[i][e]));
        ss = fmaf(h, h, ss);
        uh = fmaf(u[j][e] * w[j][e], h, uh);
      }
    }
    row_sum2<LANES>(ss, uh, red + turn);
    // (lanes without a row hold zeros, whose 1 / sqrt(0) without eps must not reach dw)
    const float r = live ? rsqrt_f(ss * a.inv_d + a.eps) : 0.f;
    const float mean = uh * r * a.inv_d;   // mean(u (.) n)
    if (kTwice) asm volatile("" ::: "memory");   // the second loads stay loads
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * LANES + l) * V, j = i % kHeld;
      float add[V], dx[V];
      if (res != nullptr) load_row<V>(res, c, D, add);
      if (kTwice) factors(i);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float n = to_f(static_cast<IO>(hr[i][e])) * r;
        dw[i][e] = fmaf(u[j][e], n, dw[i][e]);
        dx[e] = r * (u[j][e] * w[j][e] - n * mean);
        if (res != nullptr) dx[e] += add[e];
        if (kGate) dz[j][e] *= n;
      }
      store_row<V>(static_cast<IO *>(a.dx) + row * a.D, c, D, dx);
      if (kGate) store_row<V>(static_cast<IO *>(a.dz) + row * a.D, c, D, dz[j]);
    }
  }
  if (a.part == nullptr) return;
  float *part = a.part + static_cast<long long>(blockIdx.x) * a.D;
  if constexpr (R == 1) {
#pragma unroll
    for (int i = 0; i < IT; ++i) store_row<V>(part, (i * LANES + l) * V, a.D, dw[i]);
  } else {   // the rows' lanes hold the same columns: added in their order
    __shared__ float sums[R][LANES * V];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < V; ++e) sums[sub][l * V + e] = dw[i][e];
      __syncthreads();
      for (int c = threadIdx.x; c < LANES * V; c += 256) {
        float t = 0.f;
        for (int k = 0; k < R; ++k) t += sums[k][c];
        if (i * LANES * V + c < a.D) part[i * LANES * V + c] = t;
      }
    }
  }
}

// dw[c] = sum of part[g][c]: 16 columns a workgroup, 64 threads a column, each a run of groups
constexpr int kDwRuns = 64;
__global__ __launch_bounds__(16 * kDwRuns) void dw_kernel(const float *part, float *dw, int groups, int D) {
  __shared__ float sums[kDwRuns][17];
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), k = threadIdx.x >> 4;
  float t = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int g = k; g < groups; g += kDwRuns) t += part[static_cast<long long>(g) * D + c];
  }
  sums[k][threadIdx.x & 15] = t;
  __syncthreads();
  if (k < 4) {
    t = 0.f;
#pragma unroll
    for (int j = 0; j < kDwRuns / 4; ++j) t += sums[k * (kDwRuns / 4) + j][threadIdx.x & 15];
    // four lane groups of one wave
    t += __shfl_xor(t, 16, 64);
    t += __shfl_xor(t, 32, 64);
    if (k == 0 && c < D) dw[c] = t;
  }
}

// Lanes of a row and loads of a lane, the first of these that hold nv loads: short rows share a
// wave, and three loads a lane stand between the powers of two.  (16 lanes for rows of 64 bf16 channels:
// 3.9 TB/s, 8 lanes 6.1; 64 lanes for 300 channels: 3.3 TB/s and 2.2 for the gradient, 16 lanes with
// three loads 4.7 and 3.0.)
template <int LANES, int IT> struct Split { static constexpr int kLanes = LANES, kIt = IT; };
template <typename IO, typename F> auto by_width(int nv, F &&f) {
  if (nv <= 8) return f(Split<8, 1>());
  if (nv <= 16) return f(Split<16, 1>());
  if (nv <= 32) return f(Split<32, 1>());
  if (nv <= 48) return f(Split<16, 3>());
  if (nv <= 64) return f(Split<64, 1>());
  if (nv <= 96) return f(Split<32, 3>());
  if (nv <= 128) return f(Split<64, 2>());
  if (nv <= 192) return f(Split<64, 3>());
  if (nv <= 256) return f(Split<256, 1>());
  if (nv <= 384) return f(Split<128, 3>());
  if (nv <= 512) return f(Split<256, 2>());
  if (nv <= 768) return f(Split<256, 3>());
  if (nv <= 1024) return f(Split<512, 2>());
  if (nv <= 1536) return f(Split<512, 3>());
  if constexpr (sizeof(IO) == 4)   // 16384 fp32 channels; 16-bit ones are at most 2048 loads
    if (nv > 2048) return f(Split<1024, 4>());
  return f(Split<1024, 2>());
}

// The gradient's: in 16 bits one load a lane with up to 1024 lanes, whose registers leave four waves a
// SIMD (4096 channels: 4.7 TB/s with 256 lanes and two loads, 5.1 with 512; gated 4.3 and 5.1; 7001
// channels 2.7 and 3.2, gated 2.5 and 3.6; 1024 channels gated 5.0 with 64 lanes, 5.3 with 128).
// Lane counts between the powers of two gained nothing (320 lanes for 2304 channels, gated: 2.9
// TB/s against 3.4 with 512: their waves do not fill the SIMDs evenly).
template <typename IO, typename F> auto by_width_bwd(int nv, F &&f) {
  if constexpr (sizeof(IO) == 2) {
    if (nv > 96 && nv <= 128) return f(Split<128, 1>());
    if (nv > 256 && nv <= 512) return f(Split<512, 1>());
    if (nv > 512 && nv <= 1024) return f(Split<1024, 1>());
  }
  return by_width<IO>(nv, f);
}

int row_loads(int D, int io_dtype) {
  const int v = io_dtype == GDR_F32 ? 4 : 8;
  return (D + v - 1) / v;
}

template <typename IO> hipError_t fwd_io(const NormArgs &a, int nv, hipStream_t s) {
  return by_width<IO>(nv, [&](auto split) {
    constexpr int L = split.kLanes, T = threads_of(L), R = T / L;
    hipLaunchKernelGGL((norm_kernel<IO, L, split.kIt>), dim3((a.rows + R - 1) / R), dim3(T), 0, s, a);
    return hipGetLastError();
  });
}

template <typename IO> hipError_t bwd_io(const NormArgs &a, int nv, hipStream_t s) {
  return by_width_bwd<IO>(nv, [&](auto split) {
    constexpr int L = split.kLanes, I = split.kIt, T = threads_of(L);
    if (a.z != nullptr)
      hipLaunchKernelGGL((norm_bwd_kernel<IO, L, I, true>), dim3(a.groups), dim3(T), 0, s, a);
    else
      hipLaunchKernelGGL((norm_bwd_kernel<IO, L, I, false>), dim3(a.groups), dim3(T), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs &a, int io_dtype, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const int nv = row_loads(a.D, io_dtype);
  return io_dtype == GDR_BF16 ? fwd_io<uint16_t>(a, nv, s)
         : io_dtype == GDR_F16 ? fwd_io<_Float16>(a, nv, s) : fwd_io<float>(a, nv, s);
}

int rms_norm_bwd_groups(int rows, int D, int io_dtype) {
  // as many workgroups as run at once on 256 CUs: they hide each other's loads, and more would only
  // leave more parts of dw to add (the split depends on the loads and the type's size alone)
  const auto groups = [&](auto split, int vec) {
    const int T = threads_of(split.kLanes), R = T / split.kLanes;
    const int blocks = (rows - 1) / R + 1, most = 256 * (4 * bwd_waves(split.kLanes, split.kIt, vec) / (T / 64));
    return rows == 0 ? 0 : blocks < most ? blocks : most;
  };
  const int nv = row_loads(D, io_dtype);
  return io_dtype == GDR_F32 ? by_width_bwd<float>(nv, [&](auto split) { return groups(split, 4); })
                             : by_width_bwd<uint16_t>(nv, [&](auto split) { return groups(split, 8); });
}

hipError_t launch_rms_norm_bwd(const NormArgs &a, int io_dtype, hipStream_t s) {
  const int nv = row_loads(a.D, io_dtype);
  if (a.rows > 0) {
    const hipError_t e = io_dtype == GDR_BF16 ? bwd_io<uint16_t>(a, nv, s)
                         : io_dtype == GDR_F16 ? bwd_io<_Float16>(a, nv, s) : bwd_io<float>(a, nv, s);
    if (e != hipSuccess) return e;
  }
  if (a.dw != nullptr) {
    hipLaunchKernelGGL(dw_kernel, dim3((a.D + 15) / 16), dim3(16 * kDwRuns), 0, s, a.part, a.dw, a.groups, a.D);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace gdr
