// decay_step.cu -- linear attention with one decay per head, one token per
// sequence (the recurrent form, for decoding):
//   S = lambda S + k^T v (in place),  o = scale q S,   S [d_k][d_v] fp32
// The state's bytes bound it: each is read once and written once.  One block per
// (row, head) holds up to 64 rows' worth of 16-byte loads per column group in
// flight: thread = (4 value channels, one of RL key-channel lanes), 16 key rows
// of a lane at a time in registers.  Everything is fp32; only o is rounded.  lambda
// is applied as hi + lo, as the prompt form does: a rounded one, off by up to
// 2^-25 the same way at every token, would take the state 1e-4 off in 4000 tokens,
// where the roundings of the states, which go either way, leave 3e-6.
// 253 rows, 16 heads of 128/128 (535 MB): 85 to 88 us, 6.1 TB/s, 93% of the measured copy;
// one row of 6 heads of 32/64: 2.5 us on the device, back to back in a graph.
#include <cuda_bf16.h>

#include "decay_attn.h"
#include "sm100.cuh"

namespace dig {

void set_last_error(const char* msg);  // dig_api.cu

namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 256;
constexpr int kBatch = 16;  // key rows a thread has in flight

struct StepArgs {
  const void *q, *k, *v;
  long long qs, ks, vs;  // elements between rows
  const float* g;
  float scale;
  float* S;
  const int* slots;
  int n_slots;
  void* o;
  int B, H, dk, dv;
  unsigned int* status;
};

template <typename T, typename TO>
__global__ void __launch_bounds__(kThreads) decay_step_kernel(const StepArgs a) {
  __shared__ float sk[kMaxD], sq[kMaxD];
  __shared__ float4 part[kThreads];
  __shared__ float2 slam;
  const int h = blockIdx.x % a.H, b = blockIdx.x / a.H;
  const int G = a.dv >> 2, RL = kThreads / G;  // column groups, key-channel lanes
  const int cg = threadIdx.x % G, rl = threadIdx.x / G;
  const bool on = rl < RL;
  griddep_wait();
  griddep_launch_dependents();
  const int slot = a.slots ? a.slots[b] : b;
  if (slot < 0) return;  // a padding row
  if (slot >= a.n_slots) {
    if (threadIdx.x == 0 && h == 0 && a.status) set_status(a.status, DIG_ERR_INVALID_ARGUMENT);
    return;
  }
  float* S = a.S + ((size_t)slot * a.H + h) * a.dk * a.dv + 4 * cg;
  float4 s[kBatch];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * RL;
      if (on && r < a.dk) s[i] = *reinterpret_cast<const float4*>(S + (size_t)r * a.dv);
    }
  };
  load(rl);
  const T* q = static_cast<const T*>(a.q) + b * a.qs + (size_t)h * a.dk;
  const T* k = static_cast<const T*>(a.k) + b * a.ks + (size_t)h * a.dk;
  const T* vp = static_cast<const T*>(a.v) + b * a.vs + (size_t)h * a.dv;
  if (threadIdx.x < a.dk) {
    sk[threadIdx.x] = static_cast<float>(k[threadIdx.x]);
    sq[threadIdx.x] = static_cast<float>(q[threadIdx.x]);
  }
  float v[4];
  load_row<4>(vp + 4 * cg, v);
  if (threadIdx.x == kThreads - 1) slam = decay_pow(a.g[h], 1);
  // a slot that an earlier row of the call has belongs to that row
  int taken = 0;
  if (a.slots)
    for (int j = threadIdx.x; j < b; j += kThreads) taken |= a.slots[j] == slot;
  if (__syncthreads_or(taken)) {
    if (threadIdx.x == 0 && h == 0 && a.status) set_status(a.status, DIG_ERR_INVALID_ARGUMENT);
    return;
  }
  const float lam = slam.x, low = slam.y;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r0 = rl; r0 < a.dk; r0 += kBatch * RL) {
    if (r0 != rl) load(r0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * RL;
      if (on && r < a.dk) {
        const float kr = sk[r], qr = sq[r];
        s[i].x = fmaf(lam, s[i].x, fmaf(low, s[i].x, kr * v[0]));
        s[i].y = fmaf(lam, s[i].y, fmaf(low, s[i].y, kr * v[1]));
        s[i].z = fmaf(lam, s[i].z, fmaf(low, s[i].z, kr * v[2]));
        s[i].w = fmaf(lam, s[i].w, fmaf(low, s[i].w, kr * v[3]));
        acc.x = fmaf(qr, s[i].x, acc.x);
        acc.y = fmaf(qr, s[i].y, acc.y);
        acc.z = fmaf(qr, s[i].z, acc.z);
        acc.w = fmaf(qr, s[i].w, acc.w);
        *reinterpret_cast<float4*>(S + (size_t)r * a.dv) = s[i];
      }
    }
  }
  part[threadIdx.x] = acc;
  __syncthreads();
  if (rl == 0) {
    for (int i = 1; i < RL; ++i) {
      const float4 p = part[i * G + cg];
      acc.x += p.x, acc.y += p.y, acc.z += p.z, acc.w += p.w;
    }
    const float o[4] = {a.scale * acc.x, a.scale * acc.y, a.scale * acc.z, a.scale * acc.w};
    store_row<4>(static_cast<TO*>(a.o) + ((size_t)b * a.H + h) * a.dv + 4 * cg, o);
  }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

dig_status step_fail(dig_status s, const char* msg) {
  set_last_error(msg);
  return s;
}

}  // namespace
}  // namespace dig

using namespace dig;

extern "C" dig_status dig_decay_attn_step(const void* q, const void* k, const void* v, long long q_stride,
                                          long long k_stride, long long v_stride, const float* log_decay, float scale,
                                          float* S, const int* slots, int n_slots, void* o, int B, int H, int d_k,
                                          int d_v, int dtype, int out_dtype, unsigned int* device_status,
                                          void* stream) {
  if (B < 0 || H <= 0 || d_k <= 0 || d_v <= 0 || n_slots < 0)
    return step_fail(DIG_ERR_INVALID_ARGUMENT, "decay attention step: negative or zero size");
  if (d_k % 4 || d_v % 4 || d_k > kMaxD || d_v > kMaxD)
    return step_fail(DIG_ERR_UNSUPPORTED, "decay attention step: d_k and d_v must be multiples of 4 up to 256");
  if ((dtype != DIG_F32 && dtype != DIG_BF16) || (out_dtype != DIG_F32 && out_dtype != DIG_BF16))
    return step_fail(DIG_ERR_INVALID_ARGUMENT, "decay attention step: dtype / out_dtype not DIG_F32 or DIG_BF16");
  if (q_stride < (long long)H * d_k || k_stride < (long long)H * d_k || v_stride < (long long)H * d_v)
    return step_fail(DIG_ERR_INVALID_ARGUMENT, "decay attention step: a row stride is below the row's size");
  if (q_stride % 4 || k_stride % 4 || v_stride % 4)
    return step_fail(DIG_ERR_UNSUPPORTED, "decay attention step: row strides must be multiples of 4");
  if (!slots && n_slots < B)
    return step_fail(DIG_ERR_INVALID_ARGUMENT, "decay attention step: fewer states than rows");
  if ((long long)B * H > 2147483647ll) return step_fail(DIG_ERR_INVALID_ARGUMENT, "decay attention step: too many rows");
  if (B == 0) return DIG_OK;
  if (!q || !k || !v || !log_decay || !S || !o)
    return step_fail(DIG_ERR_INVALID_ARGUMENT, "decay attention step: q, k, v, log_decay, S and o must be non-NULL");
  const uintptr_t four = dtype == DIG_BF16 ? 7 : 15;  // bytes of four elements, less one
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & four)
    return step_fail(DIG_ERR_MISALIGNED, "decay attention step: q, k or v is not aligned to four elements");
  if (!al16(S) || !al16(o))
    return step_fail(DIG_ERR_MISALIGNED, "decay attention step: a tensor pointer is not 16-byte aligned");
  const StepArgs a{q, k, v, q_stride, k_stride, v_stride, log_decay, scale, S, slots, n_slots, o, B, H, d_k, d_v,
                   device_status};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)(B * (long long)H));
  using bf = __nv_bfloat16;
  auto kern = dtype == DIG_BF16 ? (out_dtype == DIG_BF16 ? decay_step_kernel<bf, bf> : decay_step_kernel<bf, float>)
                                : (out_dtype == DIG_BF16 ? decay_step_kernel<float, bf> : decay_step_kernel<float, float>);
  const cudaError_t e = launch_pdl(kern, grid, dim3(kThreads), 0, s, a);
  return e == cudaSuccess ? DIG_OK : step_fail(DIG_ERR_CUDA, cudaGetErrorString(e));
}
