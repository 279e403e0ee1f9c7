// decay_attn.cu -- the C ABI of the head-decay linear attention's prompt form and
// of its backward: argument checks, the cut of the sequences into segments, the
// workspace, launches.
#include <cstdio>
#include <cstring>

#include "decay_attn.h"
#include "sm100.cuh"
#include "tmap.h"

namespace dig {

void set_last_error(const char* msg);       // dig_api.cu
unsigned long long spin_limit_ns();         // dig_api.cu

namespace {

constexpr int kSms = 148;
// The workspace: header, the blocks' flags (in one place for every call that uses it, since calls leave them zero), states.
constexpr size_t kWsStates = 2048;
static_assert(sizeof(WsHeader) + 2 * kSms * sizeof(uint32_t) <= kWsStates, "a flag for each block");

struct Cut {
  int D;          // the kernels' padded head dim
  int seg;        // tokens of a segment
  int nps;        // segments of a sequence of L tokens (whole sequences only)
  int total;      // segment slots of the call
  int kept;       // segment states of a problem and head
  bool multi;     // whether a sequence may have several segments
  size_t states;  // floats of all problems' segment states
};

int up(long long x, int m) { return (int)((x + m - 1) / m * m); }

// How long the segments are.  One per sequence needs one pass over the data; more
// of them fill the GPU where there are few sequences, at the price of a first pass
// over k and v (about half of the second pass's bytes) and of joining the earlier
// segments' states (about a seventh of a chunk's time each, at 128 x 128).  Whole
// sequences: the cheapest count by that reckoning.  Packed ones, whose lengths the
// host does not know: two segments' worth of work per SM.
Cut cut_of(int B, int H, int L, int dk, int dv, int chunk, int per_sm, bool packed, int nprob) {
  Cut r{};
  r.D = (dk > 64 || dv > 64) ? 128 : 64;
  const int slots = kSms * per_sm;
  if (packed) {
    const long long share = (long long)L * H * nprob / (2 * slots);
    r.seg = up(share < 1 ? 1 : (share > (1 << 30) ? (1 << 30) : share), chunk);
    r.total = B + L / r.seg;
    r.nps = 1;
    r.multi = L > r.seg;
    // sequences of one segment have none, and one of n > seg tokens has at most 2 (n / seg)
    r.kept = 2ll * (L / r.seg) < r.total ? 2 * (L / r.seg) : r.total;
  } else {
    double best = 0;
    const int most = L > 0 ? (L + chunk - 1) / chunk : 1;
    for (int n = 1; n <= most && n <= 512; ++n) {
      const int seg = up(L > 0 ? (L + n - 1) / n : 1, chunk);
      const int ns = L > 0 ? (L + seg - 1) / seg : 1;
      const long long units = (long long)B * H * nprob * ns;
      const double waves = (double)((units + slots - 1) / slots);
      const double cost = waves * (seg / chunk + 1) * (ns > 1 ? 1.5 : 1.0) + (ns > 1 ? 1.0 + 0.15 * (ns - 1) : 0.0);
      if (n == 1 || cost < best) {
        best = cost;
        r.seg = seg;
        r.nps = ns;
      }
    }
    r.total = B * r.nps;
    r.kept = r.total;
    r.multi = r.nps > 1;
  }
  r.states = r.multi ? (size_t)nprob * r.kept * H * r.D * r.D : 0;
  return r;
}

dig_status attn_fail(dig_status s, const char* msg) {
  char buf[256];
  snprintf(buf, sizeof(buf), "decay attention: %s", msg);
  set_last_error(buf);
  return s;
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Tokens are read in pieces of four elements (eight where all of a tensor's tokens allow it).
bool al4(const void* p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == DIG_BF16 ? 7u : 15u)) == 0; }

// Sizes a kernel can address: rows and segment slots in int, elements in 2^40.
bool size_ok(int B, int H, int L, int d_k, int d_v, bool packed) {
  const long long rows = packed ? L : (long long)B * L;
  return rows <= 2147483647ll - 256 && rows * H * (d_k > d_v ? d_k : d_v) < (1ll << 40) && (long long)B + L <= 2147483647ll &&
         H <= 65535;
}

// bf16 in and out runs on the tensor core (chunks of 128 tokens), the rest on the FP32 pipes (chunks of 32).
bool on_tc(int dtype, int out_dtype) { return dtype == DIG_BF16 && out_dtype == DIG_BF16; }

Cut cut_for(int B, int H, int L, int dk, int dv, bool packed, int nprob) {
  return cut_of(B, H, L, dk, dv, 32, dk <= 64 && dv <= 64 ? 3 : 2, packed, nprob);
}

// How the tensor-core kernel's chunks are dealt.  Costs in chunks of a block's time:
//   - uncut units: the most that one block gets of them;
//   - cut, one pass (the blocks hand states on): the run, and half of it again where a unit spans more than two blocks
//     (their parts are walked for the state first), some 2.5 for starts and waits, a tenth for each state joined.
//     Backward of 4 x 4096 tokens, 16 heads of 128/128, 192 units on 148 blocks: 215 us, uncut 257, in two passes 281;
//     7 packed prompts of 16382 tokens, 16 heads of 128/128: 115 us, in two passes 124; 2 x 12544 tokens, 6 heads of
//     32/64, 25 blocks to a unit: 54 us, in two passes 60;
//   - cut, two passes with a kernel between that joins the states, where a unit has 32 blocks and more: joining would cost
//     each block more than the two launches do (16384 tokens, 2 heads of 128/128, 64 blocks: 37 us, joined by the blocks
//     of the second pass 50; 8192, 4 of 64/64: 28 and 31; 4096, one of 64/64, 32 blocks: 24.5 and 25.4).
// Packed sequences, whose lengths the host does not know, are taken to be alike and always dealt by the chunk.
struct Deal {
  DecayDeal d;
  int D;
  size_t states;  // floats
};
Deal deal_for(int B, int H, int L, int dk, int dv, bool packed, int nprob) {
  Deal r{};
  r.D = dk <= 64 && dv <= 64 ? 64 : 128;
  const long long slots = (long long)kSms * (r.D == 64 ? 2 : 1);
  const long long units = (long long)B * H * nprob;
  const int n = packed ? (int)(((long long)L / 128 + B) / (B > 0 ? B : 1)) : (L > 128 ? (L + 127) / 128 : 1);
  const long long total = units * (n > 0 ? n : 1);
  r.d = DecayDeal{(int)(units < slots ? units : slots), n, n, nprob, 0, 0};
  const bool cuttable = packed ? L > 128 : n > 1;
  double best = (double)((units + r.d.grid - 1) / r.d.grid) * n;
  if (cuttable && packed) {
    r.d.grid = (int)(total < slots ? total : slots);
    r.d.handoff = 1;
  } else if (cuttable) {
    for (long long c = (total + slots - 1) / slots, k = 0; k < 64 && (k == 0 || c <= n); ++c, ++k) {
      const int grid = (int)(k == 0 && total >= slots ? slots : (total + c - 1) / c);
      const double per_unit = (double)n * grid / total;  // blocks
      const bool two = per_unit >= 32;
      const double cost = c + (two ? 0.42 * c + 3.0 : (per_unit <= 1.0 ? 1.0 : 0.45 * c + 2.5 + 0.1 * per_unit));
      if (cost < best) {
        best = cost;
        r.d.grid = grid;
        r.d.gran = 1;
        r.d.handoff = !two;
      }
    }
  }
  if (packed) r.d.gran = 1;
  r.d.joined = cuttable && r.d.gran == 1 && !r.d.handoff;
  r.states = r.d.handoff || r.d.joined ? (size_t)2 * r.d.grid * r.D * r.D : 0;
  return r;
}

// The checks that the forward and the backward share.
dig_status check(const void* q, const void* k, const void* v, long long qs, long long ks, long long vs, const float* g,
                 const int* cu, int B, int H, int L, int d_k, int d_v, int grid_h, int grid_w, int mode, int dtype,
                 int out_dtype, const void* ws, size_t ws_bytes, int pass) {
  if (B < 0 || H <= 0 || L < 0 || d_k <= 0 || d_v <= 0) return attn_fail(DIG_ERR_INVALID_ARGUMENT, "negative or zero size");
  if (!cu && (grid_h < 0 || grid_w < 0 || (long long)grid_h * grid_w != L))
    return attn_fail(DIG_ERR_INVALID_ARGUMENT, "L is not grid_h * grid_w");
  if (mode < 0 || mode > (cu ? DIG_SCAN_ROW_REV : DIG_SCAN_COL_REV))
    return attn_fail(DIG_ERR_INVALID_ARGUMENT, cu ? "packed sequences are scanned in ROW_FWD or ROW_REV order"
                                                  : "scan_mode not in 0..3");
  if ((dtype != DIG_F32 && dtype != DIG_BF16) || (out_dtype != DIG_F32 && out_dtype != DIG_BF16))
    return attn_fail(DIG_ERR_INVALID_ARGUMENT, "dtype / out_dtype not DIG_F32 or DIG_BF16");
  if (d_k % 4 || d_v % 4 || d_k > 128 || d_v > 128)
    return attn_fail(DIG_ERR_UNSUPPORTED, "d_k and d_v must be multiples of 4 up to 128");
  if (qs < (long long)H * d_k || ks < (long long)H * d_k || vs < (long long)H * d_v)
    return attn_fail(DIG_ERR_INVALID_ARGUMENT, "a token stride is below the token's size");
  if (qs % 4 || ks % 4 || vs % 4) return attn_fail(DIG_ERR_UNSUPPORTED, "token strides must be multiples of 4");
  if (!size_ok(B, H, L, d_k, d_v, cu != nullptr)) return attn_fail(DIG_ERR_INVALID_ARGUMENT, "tensor too large");
  if (B == 0) return DIG_OK;
  if (!g || !ws) return attn_fail(DIG_ERR_INVALID_ARGUMENT, "log_decay and the workspace must be non-NULL");
  if (L > 0 && (!q || !k || !v)) return attn_fail(DIG_ERR_INVALID_ARGUMENT, "q, k and v must be non-NULL");
  if (!al4(q, dtype) || !al4(k, dtype) || !al4(v, dtype))
    return attn_fail(DIG_ERR_MISALIGNED, "q, k or v is not aligned to four elements");
  if (!al16(ws)) return attn_fail(DIG_ERR_MISALIGNED, "the workspace is not 16-byte aligned");
  if (ws_bytes < dig_decay_attn_workspace_bytes(B, H, L, d_k, d_v, dtype, cu != nullptr, pass))
    return attn_fail(DIG_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  return DIG_OK;
}

// Maps of the call's tensors for the TMA, where alignment and the scan allow them: whole rows of tokens in the row
// orders (and where the grid is one row or column), runs of 16 tokens of a column in the column orders.
struct MapSource {
  const void* base;
  int d;
  long long stride;
};
void encode_maps(DecayArgs& a, const MapSource* t, int n, const MapSource* o, int no, int mode) {
  a.fetch = kFetchTokens;
  const bool rows = a.cu || mode < 2 || a.Hg == 1 || a.Wg == 1;
  if (a.L == 0 || (!rows && a.Hg % kColRun) || !tmap_available()) return;
  for (int i = 0; i < n + no; ++i) {
    const MapSource& m = i < n ? t[i] : o[i - n];
    if (!al16(m.base) || m.d % 8 || m.stride % 8) return;
    const uint64_t st = (uint64_t)m.stride, L = (uint64_t)a.L;
    const uint64_t len[2][3] = {{L, a.cu ? 1u : (uint64_t)a.B, 1}, {(uint64_t)a.Hg, (uint64_t)a.Wg, (uint64_t)a.B}};
    const uint64_t stride[2][3] = {{st, L * st, L * st}, {st * (uint64_t)a.Wg, st, L * st}};
    const uint32_t box = rows ? 128 : kColRun;
    if (!tmap_heads(i < n ? &a.map[i] : &a.omap[i - n], m.base, m.d, a.H, len[!rows], stride[!rows], box)) return;
  }
  a.fetch = rows ? kFetchRows : kFetchCols;
}

dig_status launch(DecayArgs& a, int nprob, int dk, int dv, void* ws, int dtype, int out_dtype, cudaStream_t s) {
  a.segst = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsStates);
  a.status = &static_cast<WsHeader*>(ws)->status;
  cudaError_t e;
  if (on_tc(dtype, out_dtype)) {
    const Deal d = deal_for(a.B, a.H, a.L, dk, dv, a.cu != nullptr, nprob);
    a.deal = d.d;
    a.flag = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + sizeof(WsHeader));
    a.counter = static_cast<WsHeader*>(ws)->pad;
    const unsigned long long limit = spin_limit_ns();
    a.short_wait = limit != 0 && limit < kSpinLimitNs;
    a.late_chunk = limit < 1000 ? (int)limit - 1 : -1;
    e = launch_decay_tc(a, d.D, s);
  } else {
    const Cut c = cut_for(a.B, a.H, a.L, dk, dv, a.cu != nullptr, nprob);
    a.seg = c.seg;
    a.nps = c.nps;
    a.states = c.kept;
    a.segst_problem = (long long)c.kept * a.H * c.D * c.D;
    e = launch_decay_f32(a, nprob, c.total, c.multi, c.D, dtype, out_dtype, s);
  }
  return e == cudaSuccess ? DIG_OK : attn_fail(DIG_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace
}  // namespace dig

using namespace dig;

extern "C" {

size_t dig_decay_attn_workspace_bytes(int B, int H, int L, int d_k, int d_v, int dtype, int packed, int pass) {
  if (B < 0 || H <= 0 || L < 0 || d_k <= 0 || d_v <= 0 || d_k > 128 || d_v > 128 || d_k % 4 || d_v % 4 ||
      (pass != 0 && pass != 1) || (dtype != DIG_F32 && dtype != DIG_BF16) || !size_ok(B, H, L, d_k, d_v, packed != 0))
    return 0;
  size_t n = cut_for(B, H, L, d_k, d_v, packed != 0, pass ? 3 : 1).states;
  if (dtype == DIG_BF16) {  // either output type
    const size_t m = deal_for(B, H, L, d_k, d_v, packed != 0, pass ? 3 : 1).states;
    n = m > n ? m : n;
  }
  return kWsStates + n * sizeof(float);
}

dig_status dig_decay_attn_fwd(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                              long long v_stride, const float* log_decay, float scale, const int* cu_seqlens,
                              const float* S0, float* S_final, const int* slots, int n_slots, void* o, int B, int H,
                              int L, int d_k, int d_v, int grid_h, int grid_w, int scan_mode, int dtype, int out_dtype,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const dig_status st = check(q, k, v, q_stride, k_stride, v_stride, log_decay, cu_seqlens, B, H, L, d_k, d_v, grid_h,
                              grid_w, scan_mode, dtype, out_dtype, workspace, workspace_bytes, 0);
  if (st != DIG_OK || B == 0) return st;
  if (slots && n_slots < 0) return attn_fail(DIG_ERR_INVALID_ARGUMENT, "n_slots must be >= 0");
  if (L > 0 && !o) return attn_fail(DIG_ERR_INVALID_ARGUMENT, "o must be non-NULL");
  if (!al16(o) || !al16(S0) || !al16(S_final)) return attn_fail(DIG_ERR_MISALIGNED, "a tensor pointer is not 16-byte aligned");
  DecayArgs a{};
  a.g = log_decay;
  a.cu = cu_seqlens;
  a.slots = (S0 || S_final) ? slots : nullptr;
  a.n_slots = n_slots;
  a.B = B, a.H = H, a.L = L, a.Hg = grid_h, a.Wg = grid_w;
  a.p[0] = DecayProblem{q, k, v, o, q_stride, k_stride, v_stride, S0, S_final, d_k, d_v, 0, 0, scan_mode, scale, 1.f, scale, 0, 1, 2};
  if (on_tc(dtype, out_dtype)) {
    const MapSource t[3] = {{q, d_k, q_stride}, {k, d_k, k_stride}, {v, d_v, v_stride}};
    const MapSource to[1] = {{o, d_v, (long long)H * d_v}};
    encode_maps(a, t, 3, to, 1, scan_mode);
  }
  return launch(a, 1, d_k, d_v, workspace, dtype, out_dtype, static_cast<cudaStream_t>(stream));
}

dig_status dig_decay_attn_bwd(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                              long long v_stride, const float* log_decay, float scale, const int* cu_seqlens,
                              const float* S0, const void* dO, const float* dS_final, void* dq, void* dk, void* dv,
                              float* dS0, int B, int H, int L, int d_k, int d_v, int grid_h, int grid_w, int scan_mode,
                              int dtype, int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const dig_status st = check(q, k, v, q_stride, k_stride, v_stride, log_decay, cu_seqlens, B, H, L, d_k, d_v, grid_h,
                              grid_w, scan_mode, dtype, out_dtype, workspace, workspace_bytes, 1);
  if (st != DIG_OK || B == 0) return st;
  if (L > 0 && (!dO || !dq || !dk || !dv)) return attn_fail(DIG_ERR_INVALID_ARGUMENT, "dO, dq, dk and dv must be non-NULL");
  if (!al16(dO) || !al16(dq) || !al16(dk) || !al16(dv) || !al16(S0) || !al16(dS_final) || !al16(dS0))
    return attn_fail(DIG_ERR_MISALIGNED, "a tensor pointer is not 16-byte aligned");
  DecayArgs a{};
  a.g = log_decay;
  a.cu = cu_seqlens;
  a.B = B, a.H = H, a.L = L, a.Hg = grid_h, a.Wg = grid_w;
  const long long os = (long long)H * d_v;
  const int rev = scan_mode ^ 1;
  a.p[0] = DecayProblem{dO, v, k, dq, os, v_stride, k_stride, S0, nullptr, d_v, d_k, 1, 0, scan_mode, scale, 1.f, scale, 3, 2, 1};
  a.p[1] = DecayProblem{k, q, dO, dv, k_stride, q_stride, os, dS_final, dS0, d_k, d_v, 0, 1, rev, scale, scale, 1.f, 1, 0, 3};
  a.p[2] = DecayProblem{v, dO, q, dk, v_stride, os, q_stride, dS_final, nullptr, d_v, d_k, 1, 1, rev, scale, scale, 1.f, 2, 3, 0};
  if (on_tc(dtype, out_dtype)) {
    const MapSource t[4] = {{q, d_k, q_stride}, {k, d_k, k_stride}, {v, d_v, v_stride}, {dO, d_v, os}};
    const MapSource to[3] = {{dq, d_k, (long long)H * d_k}, {dv, d_v, os}, {dk, d_k, (long long)H * d_k}};
    encode_maps(a, t, 4, to, 3, scan_mode);
  }
  return launch(a, 3, d_k, d_v, workspace, dtype, out_dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
