// layer_norm.cu -- layer norm over rows of D values and its backward
// (slide eq. (10), "LN"):
//   y  = (x - mean) rstd w + b,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  a = dy w,
//   dx = rstd (a - mean(a) - xh mean(a xh)),  dw = sum_rows dy xh,  db = sum_rows dy
// Both are memory-bound: one read of x (and dy), one write of y (dx).  A row is
// held in the registers of TPR threads, at most 16 values each (a warp up to 512
// values, 512 threads up to 8192), so the variance is the two-pass one at no extra
// traffic; rows wider than that are re-read from cache.  A thread keeps its columns
// from row to row, so weight and bias stay in registers, and asks for the next row
// before it reduces this one.  All sums are fp32.  The weight
// gradients are summed per thread over the block's rows, then over the block's
// rows of threads, and the blocks' partial rows by a second kernel, all in a
// fixed order (no atomics: the same bits from run to run).
// Forward 16384 x 4096 bf16 48 us (5.6 TB/s, 85% of the measured copy), backward 8191 x 4096 fp32 69 to 71 us
// (5.8 TB/s, 88%); rows that 16-byte vectors do not fit run at 2 to 4 TB/s (a value at a time: the loads'
// and the reductions' latency).
#include <cuda_bf16.h>

#include "../../include/dig.h"
#include "dig_common.cuh"
#include "sm100.cuh"

namespace dig {

void set_last_error(const char* msg);  // dig_api.cu

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 296;  // blocks of the backward: two per SM, one partial row of dw and db each

// V consecutive elements as fp32 (V * sizeof(T) = 16, or V = 1).
template <typename T, int V>
__device__ __forceinline__ void ld_vec(const T* p, float* f) {
  if constexpr (V == 1) {
    f[0] = static_cast<float>(*p);
  } else if constexpr (sizeof(T) == 2) {
    static_assert(V == 8, "16-byte vectors");
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(p + i));
      f[i] = u.x, f[i + 1] = u.y, f[i + 2] = u.z, f[i + 3] = u.w;
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void st_vec(T* p, const float* f) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2) *p = __float2bfloat16_rn(f[0]);
    else *p = f[0];
  } else if constexpr (sizeof(T) == 2 && V == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                              pack_bf16x2(f[6], f[7]));
  } else {
    store_row<V>(p, f);
  }
}

// V elements as they are in memory, and as fp32.
template <typename T, int V>
struct Raw {
  uint4 u;
  __device__ __forceinline__ void load(const T* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        f[i] = __uint_as_float(w[i]);
      }
    }
  }
};
template <typename T>
struct Raw<T, 1> {
  T u;
  __device__ __forceinline__ void load(const T* p) { u = *p; }
  __device__ __forceinline__ void zero() { u = static_cast<T>(0.f); }
  __device__ __forceinline__ void get(float* f) const { *f = static_cast<float>(u); }
};

template <int TPR>
constexpr int threads_of = TPR > kThreads ? TPR : kThreads;

// Sums of N values over the TPR threads of a row; every thread gets them.  `red`
// holds two sets of N floats per warp for rows of several warps, used in turn so
// that one barrier per call is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float* v, float* red, int& turn) {
  constexpr int WARPS = threads_of<TPR> / 32;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xFFFFFFFFu, v[n], m);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    float* r = red + turn * (WARPS * N);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) r[n * WARPS + warp] = v[n];
    }
    __syncthreads();
    const int w0 = warp / (TPR / 32) * (TPR / 32);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = r[n * WARPS + w0];
#pragma unroll
      for (int i = 1; i < TPR / 32; ++i) v[n] += r[n * WARPS + w0 + i];
    }
  }
}
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red, int& turn) {
  row_sums<TPR, 1>(&v, red, turn);
  return v;
}

struct LnArgs {
  const void* x;
  long long x_stride;
  const float *w, *b;
  float eps;
  void* y;
  float *mean, *rstd;
  long long rows;
  int D;
};

// Rows in registers: NV vectors of V values per thread, TPR threads per row.  Blocks an SM: three of 256 threads (80
// registers; 64 with their spills took 39 us for 33554 x 1000 bf16 values where 80 took 27, and a hundred took 55 for
// 16384 x 4096 where 80 took 48); of 512 threads two, where one took 38 us for 4096 x 8192 bf16 values and two 30.
template <typename T, typename TO, int V, int NV, int TPR>
__global__ void __launch_bounds__(threads_of<TPR>, (V == 1 ? (TPR == 512 ? 1 : 2) : TPR == 512 ? (V == 8 ? 2 : 1) : 3)) ln_fwd_kernel(const LnArgs a) {
  constexpr int NT = threads_of<TPR>, RPB = NT / TPR;
  __shared__ float red[2 * NT / 32];
  const int tr = threadIdx.x % TPR;
  int turn = 0;
  const T* x = static_cast<const T*>(a.x);
  TO* y = static_cast<TO*>(a.y);
  const float inv_d = 1.f / a.D;
  griddep_wait();
  griddep_launch_dependents();
  Raw<T, V> next[NV];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + tr) * V;
      if (row < a.rows && c < a.D) next[i].load(x + row * a.x_stride + c);
      else next[i].zero();
    }
  };
  const long long step = (long long)gridDim.x * RPB;
  long long r0 = (long long)blockIdx.x * RPB;
  fetch(r0 + threadIdx.x / TPR);
  float w[NV * V], b[NV * V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + tr) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) w[i * V + e] = 1.f, b[i * V + e] = 0.f;
    if (a.w && c < a.D) ld_vec<float, V>(a.w + c, w + i * V);
    if (a.b && c < a.D) ld_vec<float, V>(a.b + c, b + i * V);
  }
  // every thread of a block takes the same number of steps (barriers in row_sum)
  for (; r0 < a.rows; r0 += step) {
    const long long row = r0 + threadIdx.x / TPR;
    float f[NV * V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) next[i].get(f + i * V);
    fetch(row + step);
#pragma unroll
    for (int i = 0; i < NV * V; ++i) s += f[i];
    const float mean = row_sum<TPR>(s, red, turn) * inv_d;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * TPR + tr) * V < a.D) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          f[i * V + e] -= mean;
          q = fmaf(f[i * V + e], f[i * V + e], q);
        }
      }
    }
    const float rstd = rsqrtf(row_sum<TPR>(q, red, turn) * inv_d + a.eps);
    if (row >= a.rows) continue;
    if (tr == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + tr) * V;
      if (c >= a.D) continue;
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf(f[i * V + e] * rstd, w[i * V + e], b[i * V + e]);
      st_vec<TO, V>(y + row * a.D + c, o);
    }
  }
}

// Rows of any width, one block each, re-read from cache for the second and third pass.
template <typename T, typename TO>
__global__ void __launch_bounds__(kThreads) ln_fwd_wide_kernel(const LnArgs a) {
  __shared__ float red[2 * kThreads / 32];
  int turn = 0;
  const float inv_d = 1.f / a.D;
  griddep_wait();
  griddep_launch_dependents();
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    TO* y = static_cast<TO*>(a.y) + row * a.D;
    float s = 0.f;
    for (int c = threadIdx.x; c < a.D; c += kThreads) s += static_cast<float>(x[c]);
    const float mean = row_sum<kThreads>(s, red, turn) * inv_d;
    float q = 0.f;
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      const float d = static_cast<float>(x[c]) - mean;
      q = fmaf(d, d, q);
    }
    const float rstd = rsqrtf(row_sum<kThreads>(q, red, turn) * inv_d + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      const float v = fmaf((static_cast<float>(x[c]) - mean) * rstd, a.w ? a.w[c] : 1.f, a.b ? a.b[c] : 0.f);
      st_vec<TO, 1>(y + c, &v);
    }
  }
}

struct LnBwdArgs {
  const void* x;
  long long x_stride;
  const float *w, *mean, *rstd;
  const void* dy;
  void* dx;
  float *pw, *pb;  // partial rows of dw and db, [blocks][D]; NULL: not wanted
  long long rows;
  int D;
};

// Two blocks of 256 threads an SM, 128 registers, at D from 2049 to 4096: with 163 and one block 8191 x 4096 fp32 values take
// 90 us, so 70.  Elsewhere the compiler's own choice (0: no bound) is the better one.
template <typename T, typename TO, int V, int NV, int TPR>
__global__ void __launch_bounds__(threads_of<TPR>, (V > 1 && TPR == 256 ? 2 : 0)) ln_bwd_kernel(const LnBwdArgs a) {
  constexpr int NT = threads_of<TPR>, RPB = NT / TPR;
  __shared__ float red[4 * NT / 32];
  extern __shared__ float part[];  // [RPB][D], only for RPB > 1
  const int tr = threadIdx.x % TPR, rb = threadIdx.x / TPR;
  int turn = 0;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  TO* dx = static_cast<TO*>(a.dx);
  const float inv_d = 1.f / a.D;
  float gw[NV * V], gb[NV * V];
#pragma unroll
  for (int i = 0; i < NV * V; ++i) gw[i] = gb[i] = 0.f;
  griddep_wait();
  griddep_launch_dependents();
  Raw<T, V> nx[NV], ny[NV];
  float nmean, nrstd;
  auto fetch = [&](long long row) {
    const bool on = row < a.rows;
    nmean = on ? __ldg(a.mean + row) : 0.f;
    nrstd = on ? __ldg(a.rstd + row) : 0.f;  // 0: nothing of a row that is not there counts
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + tr) * V;
      if (on && c < a.D) {
        nx[i].load(x + row * a.x_stride + c);
        ny[i].load(dy + row * a.D + c);
      } else {
        nx[i].zero();
        ny[i].zero();
      }
    }
  };
  const long long step = (long long)gridDim.x * RPB;
  long long r0 = (long long)blockIdx.x * RPB;
  fetch(r0 + rb);
  float w[NV * V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + tr) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) w[i * V + e] = 1.f;
    if (a.w && c < a.D) ld_vec<float, V>(a.w + c, w + i * V);
  }
  for (; r0 < a.rows; r0 += step) {
    const long long row = r0 + rb;
    float xh[NV * V], g[NV * V];
    const float mean = nmean, rstd = nrstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      nx[i].get(xh + i * V);
      ny[i].get(g + i * V);
    }
    fetch(row + step);
    float s[2] = {0.f, 0.f};
    // Past D g and w g are 0, but xh = (0 - mean) rstd need not be finite, nor 0 times it 0.  It is not only where all values
    // of the row are the mean itself (one that is not is off by 2^-25 of it at least, and |xh| is at most sqrt(D)).  So the
    // mean of those columns is taken as 0; or, where 512 threads have no register to spare for that, the sum of such a row,
    // whose xh are all 0, is.
    constexpr bool ZERO = TPR < 512;
#pragma unroll
    for (int n = 0; n < NV * V; ++n) {
      xh[n] = (xh[n] - (ZERO && (n / V * TPR + tr) * V >= a.D ? 0.f : mean)) * rstd;
      gw[n] = fmaf(g[n], xh[n], gw[n]);
      gb[n] += g[n];
      g[n] *= w[n];
      s[0] += g[n];
      s[1] = fmaf(g[n], xh[n], s[1]);
    }
    const bool flat = !ZERO && !isfinite(mean * rstd);
    row_sums<TPR, 2>(s, red, turn);
    const float s1 = s[0] * inv_d, s2 = flat ? 0.f : s[1] * inv_d;
    if (row >= a.rows) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + tr) * V;
      if (c >= a.D) continue;
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = rstd * (g[i * V + e] - s1 - xh[i * V + e] * s2);
      st_vec<TO, V>(dx + row * a.D + c, o);
    }
  }
  // the block's partial sums: its rows of threads are added in order
  auto leave = [&](const float* v, float* out) {
    if (!out) return;
    float* p = out + (size_t)blockIdx.x * a.D;
    if constexpr (RPB == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tr) * V;
        if (c < a.D) st_vec<float, V>(p + c, v + i * V);
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tr) * V;
        if (c < a.D) st_vec<float, V>(part + (size_t)rb * a.D + c, v + i * V);
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.D; c += NT) {
        float s = part[c];
#pragma unroll
        for (int r = 1; r < RPB; ++r) s += part[(size_t)r * a.D + c];
        p[c] = s;
      }
    }
  };
  leave(gw, a.pw);
  leave(gb, a.pb);
}

// Rows of any width: one block per row at a time, re-read from cache; the block's
// weight gradients are kept in its partial rows in global memory.
template <typename T, typename TO>
__global__ void __launch_bounds__(kThreads) ln_bwd_wide_kernel(const LnBwdArgs a) {
  __shared__ float red[2 * kThreads / 32];
  int turn = 0;
  const float inv_d = 1.f / a.D;
  griddep_wait();
  griddep_launch_dependents();
  float* pw = a.pw ? a.pw + (size_t)blockIdx.x * a.D : nullptr;
  float* pb = a.pb ? a.pb + (size_t)blockIdx.x * a.D : nullptr;
  for (int c = threadIdx.x; c < a.D; c += kThreads) {  // a column stays with one thread
    if (pw) pw[c] = 0.f;
    if (pb) pb[c] = 0.f;
  }
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + row * a.D;
    TO* dx = static_cast<TO*>(a.dx) + row * a.D;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      const float g = static_cast<float>(dy[c]), xh = (static_cast<float>(x[c]) - mean) * rstd;
      if (pw) pw[c] += g * xh;
      if (pb) pb[c] += g;
      const float aw = a.w ? g * a.w[c] : g;
      s1 += aw;
      s2 = fmaf(aw, xh, s2);
    }
    s1 = row_sum<kThreads>(s1, red, turn) * inv_d;
    s2 = row_sum<kThreads>(s2, red, turn) * inv_d;
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      const float g = static_cast<float>(dy[c]), xh = (static_cast<float>(x[c]) - mean) * rstd;
      const float v = rstd * ((a.w ? g * a.w[c] : g) - s1 - xh * s2);
      st_vec<TO, 1>(dx + c, &v);
    }
  }
}

// out[c] = sum of the blocks' partial rows: 32 columns per block, kGroups groups of
// rows whose sums are added in order.  Its time is a few trips to L2, so groups are
// many and a thread's loads go out ahead of its additions.
constexpr int kGroups = 32;
__global__ void __launch_bounds__(32 * kGroups) ln_bwd_join_kernel(const float* __restrict__ pw, const float* __restrict__ pb,
                                                          float* dw, float* db, int blocks, int D) {
  __shared__ float part[kGroups][33];
  griddep_wait();
  griddep_launch_dependents();
  const float* p = blockIdx.y ? pb : pw;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < D) {
    for (int r0 = grp; r0 < blocks; r0 += 5 * kGroups) {
      float x[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) x[i] = r0 + i * kGroups < blocks ? p[(size_t)(r0 + i * kGroups) * D + c] : 0.f;
#pragma unroll
      for (int i = 0; i < 5; ++i) s += x[i];
    }
  }
  part[grp][lane] = s;
  __syncthreads();
  if (grp == 0 && c < D) {
#pragma unroll
    for (int g = 1; g < kGroups; ++g) s += part[g][lane];
    out[c] = s;
  }
}

// Blocks for `rows` rows of which a block takes `rpb` at a time.
int ln_blocks(long long rows, int rpb, int cap) {
  const long long n = (rows + rpb - 1) / rpb;
  return (int)(n < 1 ? 1 : (n < cap ? n : cap));
}
constexpr int kSms = 148;

// Blocks of the forward on an SM: as many as run at once (a block keeps its columns' weights from row to row).
int ln_per_sm(const void* kernel, int threads) {
  int n = 0;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) == cudaSuccess && n > 0 ? n : 1;
}

// Picks <V, NV, TPR> for D: 16-byte vectors where `vec` allows them, and at most 16 values per thread.
template <typename T, typename F>
cudaError_t ln_pick(int D, bool vec, F&& f) {
  constexpr int V = 16 / sizeof(T);
  auto go = [&](auto v) {
    constexpr int W = decltype(v)::value;
    using std::integral_constant;
    if (D <= 256) return f(integral_constant<int, W>{}, integral_constant<int, 8 / W>{}, integral_constant<int, 32>{});
    if (D <= 512) return f(integral_constant<int, W>{}, integral_constant<int, 16 / W>{}, integral_constant<int, 32>{});
    if (D <= 1024) return f(integral_constant<int, W>{}, integral_constant<int, 16 / W>{}, integral_constant<int, 64>{});
    if (D <= 2048) return f(integral_constant<int, W>{}, integral_constant<int, 16 / W>{}, integral_constant<int, 128>{});
    if (D <= 4096) return f(integral_constant<int, W>{}, integral_constant<int, 16 / W>{}, integral_constant<int, 256>{});
    return f(integral_constant<int, W>{}, integral_constant<int, 16 / W>{}, integral_constant<int, 512>{});
  };
  return vec ? go(std::integral_constant<int, V>{}) : go(std::integral_constant<int, 1>{});
}

template <typename T, typename TO>
cudaError_t ln_fwd_launch(const LnArgs& a, bool vec, cudaStream_t s) {
  if (a.D > 8192) return launch_pdl(ln_fwd_wide_kernel<T, TO>, dim3(ln_blocks(a.rows, 1, 8 * kSms)), dim3(kThreads), 0, s, a);
  return ln_pick<T>(a.D, vec, [&](auto v, auto nv, auto tpr) {
    constexpr int TPR = decltype(tpr)::value, NT = threads_of<TPR>;
    auto k = ln_fwd_kernel<T, TO, decltype(v)::value, decltype(nv)::value, TPR>;
    static const int per_sm = [&] { return ln_per_sm(reinterpret_cast<const void*>(k), NT); }();
    return launch_pdl(k, dim3(ln_blocks(a.rows, NT / TPR, kSms * per_sm)), dim3(NT), 0, s, a);
  });
}

// Launches the backward; *blocks is the number of partial rows it leaves.
template <typename T, typename TO>
cudaError_t ln_bwd_launch(const LnBwdArgs& a, bool vec, cudaStream_t s, int* blocks) {
  if (a.D > 8192) {
    *blocks = ln_blocks(a.rows, 1, kMaxBlocks);
    return launch_pdl(ln_bwd_wide_kernel<T, TO>, dim3(*blocks), dim3(kThreads), 0, s, a);
  }
  return ln_pick<T>(a.D, vec, [&](auto v, auto nv, auto tpr) {
    constexpr int TPR = decltype(tpr)::value, NT = threads_of<TPR>, RPB = NT / TPR;
    const size_t smem = RPB > 1 ? (size_t)RPB * a.D * 4 : 0;  // at most 16 * 256 floats
    *blocks = ln_blocks(a.rows, RPB, kMaxBlocks * kThreads / NT);
    auto k = ln_bwd_kernel<T, TO, decltype(v)::value, decltype(nv)::value, TPR>;
    return launch_pdl(k, dim3(*blocks), dim3(NT), smem, s, a);
  });
}

// Whether all of the pointers (NULL too) are multiples of `bytes`.
template <typename... P>
bool aligned(size_t bytes, const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & (bytes - 1)) == 0;
}
size_t size_of(int dtype) { return dtype == DIG_BF16 ? 2 : 4; }

dig_status ln_fail(dig_status s, const char* msg) {
  set_last_error(msg);
  return s;
}

dig_status ln_check(long long rows, int D, long long x_stride, int dtype, int out_dtype) {
  if (rows < 0 || D <= 0) return ln_fail(DIG_ERR_INVALID_ARGUMENT, "layer norm: rows must be >= 0 and D >= 1");
  if (x_stride < D) return ln_fail(DIG_ERR_INVALID_ARGUMENT, "layer norm: x_stride must be at least D");
  if ((dtype != DIG_F32 && dtype != DIG_BF16) || (out_dtype != DIG_F32 && out_dtype != DIG_BF16))
    return ln_fail(DIG_ERR_INVALID_ARGUMENT, "layer norm: dtype / out_dtype not DIG_F32 or DIG_BF16");
  // (columns are counted in int, past D by a block's step)
  if (D > (1 << 30) || rows >= (1ll << 40) / x_stride) return ln_fail(DIG_ERR_INVALID_ARGUMENT, "layer norm: tensor too large");
  return DIG_OK;
}

// Whether rows are taken in 16-byte pieces: every row of the dense tensors and of x then starts at a 16-byte boundary if
// the tensor does.
bool ln_vec(int D, long long x_stride, int dtype) {
  const int v = dtype == DIG_BF16 ? 8 : 4;
  return D <= 8192 && D % v == 0 && x_stride % v == 0;
}

}  // namespace
}  // namespace dig

using namespace dig;

extern "C" {

size_t dig_layer_norm_workspace_bytes(long long rows, int D) {
  if (rows < 0 || D <= 0) return 0;
  return (size_t)2 * (rows < kMaxBlocks ? (rows < 1 ? 1 : rows) : kMaxBlocks) * D * 4;
}

dig_status dig_layer_norm_fwd(const void* x, long long x_stride, const float* weight, const float* bias, float eps,
                              void* y, float* mean, float* rstd, long long rows, int D, int dtype, int out_dtype,
                              void* stream) {
  const dig_status st = ln_check(rows, D, x_stride, dtype, out_dtype);
  if (st != DIG_OK) return st;
  if (!(eps >= 0.f)) return ln_fail(DIG_ERR_INVALID_ARGUMENT, "layer norm: eps must be >= 0");
  if (rows == 0) return DIG_OK;
  if (!x || !y) return ln_fail(DIG_ERR_INVALID_ARGUMENT, "layer norm: x and y must be non-NULL");
  const bool vec = ln_vec(D, x_stride, dtype);
  if (!aligned(size_of(dtype), x) || !aligned(size_of(out_dtype), y) || !aligned(4, weight, bias, mean, rstd))
    return ln_fail(DIG_ERR_MISALIGNED, "layer norm: a tensor pointer is not aligned to its elements");
  if (vec && !aligned(16, x, y, weight, bias))
    return ln_fail(DIG_ERR_MISALIGNED, "layer norm: rows of 16-byte pieces, but x, y, weight or bias is not 16-byte aligned");
  const LnArgs a{x, x_stride, weight, bias, eps, y, mean, rstd, rows, D};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DIG_BF16
                            ? (out_dtype == DIG_BF16 ? ln_fwd_launch<__nv_bfloat16, __nv_bfloat16>(a, vec, s)
                                                     : ln_fwd_launch<__nv_bfloat16, float>(a, vec, s))
                            : (out_dtype == DIG_BF16 ? ln_fwd_launch<float, __nv_bfloat16>(a, vec, s)
                                                     : ln_fwd_launch<float, float>(a, vec, s));
  return e == cudaSuccess ? DIG_OK : ln_fail(DIG_ERR_CUDA, cudaGetErrorString(e));
}

dig_status dig_layer_norm_bwd(const void* x, long long x_stride, const float* weight, const float* mean,
                              const float* rstd, const void* dy, void* dx, float* dweight, float* dbias, long long rows,
                              int D, int dtype, int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const dig_status st = ln_check(rows, D, x_stride, dtype, out_dtype);
  if (st != DIG_OK) return st;
  if (rows > 0 && (!x || !mean || !rstd || !dy || !dx))
    return ln_fail(DIG_ERR_INVALID_ARGUMENT, "layer norm backward: x, mean, rstd, dy and dx must be non-NULL");
  const bool vec = ln_vec(D, x_stride, dtype);
  if (!aligned(size_of(dtype), x, dy) || !aligned(size_of(out_dtype), dx) || !aligned(4, weight, mean, rstd, dweight, dbias))
    return ln_fail(DIG_ERR_MISALIGNED, "layer norm backward: a tensor pointer is not aligned to its elements");
  if ((vec && !aligned(16, x, dy, dx, weight)) || !aligned(16, workspace))
    return ln_fail(DIG_ERR_MISALIGNED,
                   "layer norm backward: the workspace, or with rows of 16-byte pieces x, dy, dx or weight, is not 16-byte aligned");
  const bool par = dweight || dbias;
  if (par && !workspace) return ln_fail(DIG_ERR_INVALID_ARGUMENT, "layer norm backward: dweight and dbias need a workspace");
  if (par && workspace_bytes < dig_layer_norm_workspace_bytes(rows, D))
    return ln_fail(DIG_ERR_WORKSPACE_TOO_SMALL, "layer norm backward: workspace too small");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  // the partial rows: [blocks][D] of dweight, then of dbias
  const size_t half = dig_layer_norm_workspace_bytes(rows, D) / 8;
  LnBwdArgs a{x, x_stride, weight, mean, rstd, dy, dx, dweight ? part : nullptr, dbias ? part + half : nullptr, rows, D};
  int blocks = 0;
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    e = dtype == DIG_BF16 ? (out_dtype == DIG_BF16 ? ln_bwd_launch<__nv_bfloat16, __nv_bfloat16>(a, vec, s, &blocks)
                                                   : ln_bwd_launch<__nv_bfloat16, float>(a, vec, s, &blocks))
                          : (out_dtype == DIG_BF16 ? ln_bwd_launch<float, __nv_bfloat16>(a, vec, s, &blocks)
                                                   : ln_bwd_launch<float, float>(a, vec, s, &blocks));
  }
  if (e == cudaSuccess && par)
    e = launch_pdl(ln_bwd_join_kernel, dim3((D + 31) / 32, 2), dim3(32 * kGroups), 0, s, a.pw, a.pb, dweight, dbias, blocks, D);
  return e == cudaSuccess ? DIG_OK : ln_fail(DIG_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"
