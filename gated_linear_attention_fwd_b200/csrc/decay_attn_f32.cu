// decay_attn_f32.cu -- head-decay linear attention on the FP32 pipes: the kernel
// of fp32 inputs, whose products the tensor core would have to take as six pairs
// of bf16 terms each, and of fp32 outputs.
//
// One block of 256 threads walks a segment in chunks of 32 tokens.  With the
// chunk's q, k, v rows and the state S in shared memory:
//   P[t][s] = a lambda^(t-s) q_t . k_s  (s <= t),
//   o_t     = c lambda^(t+1) q_t S + sum_s P[t][s] v_s,
//   S       = lambda^n S + sum_s b lambda^(n-1-s) k_s^T v_s   (n tokens in the chunk).
// S also stays in registers (a tile per thread), so that it is read from shared
// memory only as the operand of q S.  lambda^n is applied as hi + lo: a rounded
// power, applied once a chunk, would drift over a long sequence.
//
// Shared-memory reads bound the products of 32 tokens (q S, P v: 5 reads of 16 bytes
// for 16 multiply-adds of a thread), a block's chain the small calls: 4 x 1024 tokens,
// 16 heads of 128/128, 297 us, 14.5 TFLOP/s of the recurrent form's operations (one
// block an SM, with padded rows: 347 us); 8 x 256 tokens, 6 heads of 64/64, 22 us.
#include <cuda_bf16.h>

#include "decay_attn.h"
#include "sm100.cuh"

namespace dig {

namespace {

constexpr int C = 32;

template <int D>
struct F32Cfg {
  // Rows of q, k, v in 16-byte pieces, piece c of row t at c ^ (t & 7) (consecutive rows on different banks without
  // padding: two blocks of D = 128 fit an SM).  P takes the place of q once q S is formed.
  static constexpr int Q = 0, K = C * D, V = 2 * C * D, S = 3 * C * D, PW = S + D * D;
  static constexpr int FLOATS = PW + 2 * (C + 1) + 2;
  static constexpr int SMEM = FLOATS * 4;
  static constexpr int TJ = D / 32;               // value channels per thread of an output row
  static constexpr int TC = D / 16;               // key (and value) channels of a thread's state tile
};

template <typename T>
__device__ __forceinline__ float4 ld4(const T* p) {
  float v[4];
  load_row<4>(p, v);
  return make_float4(v[0], v[1], v[2], v[3]);
}

template <typename T, typename TO, int D, bool STATES>
__global__ void __launch_bounds__(256, D == 128 ? 2 : 3) decay_f32_kernel(const __grid_constant__ DecayArgs a) {
  using F = F32Cfg<D>;
  extern __shared__ float sm[];
  const int tid = threadIdx.x, h = blockIdx.y;
  const DecayProblem& p = a.p[blockIdx.z];
  griddep_wait();
  griddep_launch_dependents();
  if (a.cu && (STATES ? false : blockIdx.x == 0 && h == 0 && blockIdx.z == 0) && tid < 32) decay_check_offsets(a);
  DecayUnit u;
  if (!decay_unit(a, blockIdx.x, u)) return;
  if (STATES && (u.nseg == 1 || u.i == u.nseg - 1)) return;  // a last segment's state is formed by the output pass
  const float g = a.g[h];
  float *sq = sm + F::Q, *sk = sm + F::K, *sv = sm + F::V, *sS = sm + F::S, *sP = sq, *pw = sm + F::PW;
  auto at = [](int t, int c) { return t * D + (((c >> 2) ^ (t & 7)) << 2); };  // piece of channel c (a multiple of four) of row t
  if (tid <= C) {
    const float2 w = decay_pow(g, tid);
    pw[tid] = w.x;
    pw[C + 1 + tid] = w.y;
  }
  // this thread's state tile: key channels c0 + i, value channels j0 + j (D = 128: two groups of four, 64 apart)
  constexpr int TC = F::TC;
  const int c0 = TC * (tid >> 4), jt = tid & 15;
  auto jcol = [&](int j) { return 4 * jt + (j & 3) + 64 * (j >> 2); };
  float S[TC][TC];
#pragma unroll
  for (int i = 0; i < TC; ++i)
#pragma unroll
    for (int j = 0; j < TC; ++j) S[i][j] = 0.f;
  if (u.i == 0) {
    if (p.S0 && u.slot >= 0 && (STATES || u.nseg == 1)) {
      const float* s0 = p.S0 + ((size_t)u.slot * a.H + h) * p.dk * p.dv;
#pragma unroll
      for (int i = 0; i < TC; ++i)
#pragma unroll
        for (int j = 0; j < TC; ++j) {
          const int c = c0 + i, jj = jcol(j);
          if (c < p.dk && jj < p.dv) S[i][j] = p.s0_t ? s0[(size_t)jj * p.dk + c] : s0[(size_t)c * p.dv + jj];
        }
    }
  }
  float* seg_base = a.segst + blockIdx.z * a.segst_problem;
  auto seg_state = [&](int i) { return seg_base + ((size_t)(u.first_state + i) * a.H + h) * (D * D); };  // of the sequence's segment i
  if (!STATES && u.nseg > 1) {
    if (u.i == 0) {  // the copy of S0 that the first pass left (S0 may be overwritten by the last segment)
      const float* s0 = seg_state(u.nseg - 1);
#pragma unroll
      for (int i = 0; i < TC; ++i)
#pragma unroll
        for (int j = 0; j < TC; j += 4) {
          const float4 x = *reinterpret_cast<const float4*>(s0 + (c0 + i) * D + jcol(j));
          S[i][j] = x.x, S[i][j + 1] = x.y, S[i][j + 2] = x.z, S[i][j + 3] = x.w;
        }
    } else {
      const float2 w = decay_pow(g, a.seg);
#pragma unroll 1
      for (int m = 0; m < u.i; ++m) {
        const float* ls = seg_state(m);
#pragma unroll
        for (int i = 0; i < TC; ++i)
#pragma unroll
          for (int j = 0; j < TC; j += 4) {
            const float4 x = *reinterpret_cast<const float4*>(ls + (c0 + i) * D + jcol(j));
            S[i][j] = fmaf(w.x, S[i][j], fmaf(w.y, S[i][j], x.x));
            S[i][j + 1] = fmaf(w.x, S[i][j + 1], fmaf(w.y, S[i][j + 1], x.y));
            S[i][j + 2] = fmaf(w.x, S[i][j + 2], fmaf(w.y, S[i][j + 2], x.z));
            S[i][j + 3] = fmaf(w.x, S[i][j + 3], fmaf(w.y, S[i][j + 3], x.w));
          }
      }
    }
  }
  if (STATES && u.i == 0) {
    float* s0 = seg_state(u.nseg - 1);  // the last segment's place is free: it leaves no state there
#pragma unroll
    for (int i = 0; i < TC; ++i)
#pragma unroll
      for (int j = 0; j < TC; j += 4)
        *reinterpret_cast<float4*>(s0 + (c0 + i) * D + jcol(j)) = make_float4(S[i][j], S[i][j + 1], S[i][j + 2], S[i][j + 3]);
  }
  const T* q = static_cast<const T*>(p.q) + (size_t)h * p.dk;
  const T* k = static_cast<const T*>(p.k) + (size_t)h * p.dk;
  const T* v = static_cast<const T*>(p.v) + (size_t)h * p.dv;
  TO* o = static_cast<TO*>(p.o) + (size_t)h * p.dv;
  const size_t os = (size_t)a.H * p.dv;

  for (int t0 = 0; t0 < u.n; t0 += C) {
    const int n = min(C, u.n - t0);
    const int e = (p.lag && u.t0 + t0 == 0) ? 1 : 0;
    __syncthreads();  // the previous chunk's operands are no longer read
    if (!STATES) {
#pragma unroll
      for (int i = 0; i < TC; ++i)
#pragma unroll
        for (int j = 0; j < TC; j += 4)
          *reinterpret_cast<float4*>(sS + (c0 + i) * D + jcol(j)) = make_float4(S[i][j], S[i][j + 1], S[i][j + 2], S[i][j + 3]);
    }
    for (int x = tid; x < C * (D / 4); x += 256) {
      const int t = x / (D / 4), c = 4 * (x % (D / 4));
      float4 fq = make_float4(0.f, 0.f, 0.f, 0.f), fk = fq, fv = fq;
      if (t < n) {
        const long long row = decay_row(a, u, p.mode, u.t0 + t0 + t);
        if (c < p.dk) {
          if (!STATES) fq = ld4(q + row * p.qs + c);
          fk = ld4(k + row * p.ks + c);
        }
        if (c < p.dv) fv = ld4(v + row * p.vs + c);
      }
      if (!STATES) *reinterpret_cast<float4*>(sq + at(t, c)) = fq;
      *reinterpret_cast<float4*>(sk + at(t, c)) = fk;
      *reinterpret_cast<float4*>(sv + at(t, c)) = fv;
    }
    __syncthreads();
    if (!STATES) {
      // P: rows tid / 16 and + 16, columns tid % 16 and + 16
      float x00 = 0.f, x10 = 0.f, x11 = 0.f;  // (above the diagonal: nothing)
      {
        const int t = tid >> 4, s = tid & 15;
#pragma unroll 4
        for (int c = 0; c < p.dk; c += 4) {
          const float4 q0 = *reinterpret_cast<const float4*>(sq + at(t, c));
          const float4 q1 = *reinterpret_cast<const float4*>(sq + at(t + 16, c));
          const float4 k0 = *reinterpret_cast<const float4*>(sk + at(s, c));
          const float4 k1 = *reinterpret_cast<const float4*>(sk + at(s + 16, c));
          x00 += q0.x * k0.x + q0.y * k0.y + q0.z * k0.z + q0.w * k0.w;
          x10 += q1.x * k0.x + q1.y * k0.y + q1.z * k0.z + q1.w * k0.w;
          x11 += q1.x * k1.x + q1.y * k1.y + q1.z * k1.z + q1.w * k1.w;
        }
      }
      constexpr int TJ = F::TJ;
      const int tb = 4 * (tid >> 5), jb = TJ * (tid & 31);
      float acc[4][TJ];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = 0.f;
      auto ldj = [&](const float* src, float* w) {
        if constexpr (TJ == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(src);
          w[0] = x.x, w[1] = x.y;
        }
      };
#pragma unroll 2
      for (int c = 0; c < p.dk; c += 4) {
        float4 qv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(sq + at(tb + i, c));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float w[TJ];
          ldj(sS + (c + x) * D + jb, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float qx = reinterpret_cast<const float*>(&qv[i])[x];
#pragma unroll
            for (int j = 0; j < TJ; ++j) acc[i][j] = fmaf(qx, w[j], acc[i][j]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = p.c * pw[tb + i + 1 - e];
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] *= w;
      }
      __syncthreads();  // q is no longer read
      {
        const int t = tid >> 4, s = tid & 15;
        sP[t * (C + 1) + s] = s <= t ? p.a * pw[t - s] * x00 : 0.f;
        sP[t * (C + 1) + s + 16] = 0.f;
        sP[(t + 16) * (C + 1) + s] = p.a * pw[t + 16 - s] * x10;
        sP[(t + 16) * (C + 1) + s + 16] = s <= t ? p.a * pw[t - s] * x11 : 0.f;
      }
      __syncthreads();
#pragma unroll 4
      for (int s = 0; s < min(C, tb + 4); ++s) {  // the warp's last row
        float w[TJ];
        ldj(sv + at(s, jb & ~3) + (jb & 3), w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = sP[(tb + i) * (C + 1) + s];
#pragma unroll
          for (int j = 0; j < TJ; ++j) acc[i][j] = fmaf(x, w[j], acc[i][j]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (tb + i < n && jb < p.dv) {
          TO* dst = o + (size_t)decay_row(a, u, p.mode, u.t0 + t0 + tb + i) * os + jb;
          if constexpr (TJ == 4) store_row<4>(dst, acc[i]);
          else if constexpr (sizeof(TO) == 4) *reinterpret_cast<float2*>(dst) = make_float2(acc[i][0], acc[i][1]);
          else *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[i][0], acc[i][1]);
        }
      }
    }
    // ---- the state after the chunk, if anything needs it
    if (!STATES && t0 + C >= u.n && !(p.Sf && u.slot >= 0 && u.i == u.nseg - 1)) break;
    const float wh = pw[n - e], wl = pw[C + 1 + n - e];
#pragma unroll
    for (int i = 0; i < TC; ++i)
#pragma unroll
      for (int j = 0; j < TC; ++j) S[i][j] = fmaf(wh, S[i][j], wl * S[i][j]);
#pragma unroll 2
    for (int s = 0; s < (c0 < p.dk ? n : 0); ++s) {
      const float w = p.b * pw[n - 1 - s];
      float kc[TC], vc[TC];
#pragma unroll
      for (int i = 0; i < TC; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(sk + at(s, c0 + i));
        kc[i] = w * x.x, kc[i + 1] = w * x.y, kc[i + 2] = w * x.z, kc[i + 3] = w * x.w;
        const float4 y = *reinterpret_cast<const float4*>(sv + at(s, jcol(i)));
        vc[i] = y.x, vc[i + 1] = y.y, vc[i + 2] = y.z, vc[i + 3] = y.w;
      }
#pragma unroll
      for (int i = 0; i < TC; ++i)
#pragma unroll
        for (int j = 0; j < TC; ++j) S[i][j] = fmaf(kc[i], vc[j], S[i][j]);
    }
  }
  if (STATES) {
    float* out = seg_state(u.i);
#pragma unroll
    for (int i = 0; i < TC; ++i)
#pragma unroll
      for (int j = 0; j < TC; j += 4)
        *reinterpret_cast<float4*>(out + (c0 + i) * D + jcol(j)) = make_float4(S[i][j], S[i][j + 1], S[i][j + 2], S[i][j + 3]);
  } else if (p.Sf && u.slot >= 0 && u.i == u.nseg - 1) {
    // dS0 = lambda G_0; an empty sequence passes its state on as it is
    const float w = p.lag && u.len > 0 ? decay_pow(g, 1).x : 1.f;
    float* out = p.Sf + ((size_t)u.slot * a.H + h) * p.dk * p.dv;
#pragma unroll
    for (int i = 0; i < TC; ++i)
#pragma unroll
      for (int j = 0; j < TC; j += 4)
        if (c0 + i < p.dk && jcol(j) < p.dv)
          *reinterpret_cast<float4*>(out + (size_t)(c0 + i) * p.dv + jcol(j)) =
              make_float4(w * S[i][j], w * S[i][j + 1], w * S[i][j + 2], w * S[i][j + 3]);
  }
}

template <typename T, typename TO, int D>
cudaError_t launch(const DecayArgs& a, int nprob, int nseg_total, bool multi, cudaStream_t s) {
  const dim3 grid(nseg_total, a.H, nprob);
  cudaError_t e;
  auto run = [&](auto kern) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F32Cfg<D>::SMEM)) != cudaSuccess) return e;
    return launch_pdl(kern, grid, dim3(256), F32Cfg<D>::SMEM, s, a);
  };
  if (multi && (e = run(decay_f32_kernel<T, TO, D, true>)) != cudaSuccess) return e;
  return run(decay_f32_kernel<T, TO, D, false>);
}

}  // namespace

cudaError_t launch_decay_f32(const DecayArgs& a, int nprob, int nseg_total, bool multi, int D, int dtype, int out_dtype,
                             cudaStream_t s) {
  using bf = __nv_bfloat16;
  auto go = [&](auto d) {
    constexpr int DD = decltype(d)::value;
    if (dtype == DIG_BF16)
      return out_dtype == DIG_BF16 ? launch<bf, bf, DD>(a, nprob, nseg_total, multi, s) : launch<bf, float, DD>(a, nprob, nseg_total, multi, s);
    return out_dtype == DIG_BF16 ? launch<float, bf, DD>(a, nprob, nseg_total, multi, s) : launch<float, float, DD>(a, nprob, nseg_total, multi, s);
  };
  return D == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

}  // namespace dig
