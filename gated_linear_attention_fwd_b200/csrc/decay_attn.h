// decay_attn.h -- what the kernels of the head-decay linear attention share:
// the problems of one call, how they are cut up among blocks, and the walk from a
// block to its part.
//
// A problem is  o_t = c lambda^(t+1) q_t S0 + a sum_{s<=t} lambda^(t-s) (q_t . k_s) v_s
// over scan positions t of a sequence, with the carried state
//   S_t = lambda S_{t-1} + b k_t^T v_t.
// The forward is one problem (a = c = scale, b = 1).  The backward is three of
// the same form: dq from (dO, v, k) and S0^T in the forward's order; dv from
// (k, q, dO) and dk from (v, dO, q) in the reversed order, where the state is the
// adjoint one, starts from dS_final (transposed for dk) without the first lambda
// ("lag"), and ends, times lambda, as dS0.
//
// On the FP32 pipes a sequence is cut into segments of `seg` tokens, each walked by
// one block in chunks.  With more than one segment per sequence a first kernel leaves
// every segment's own state contribution (segment 0: with S0 in it), and the second
// one joins those before its segment into the state it starts from.  How the
// tensor-core kernel does it is at DecayDeal.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "dig_common.cuh"

namespace dig {

struct DecayProblem {
  const void *q, *k, *v;
  void* o;
  long long qs, ks, vs;  // elements between tokens
  const float* S0;       // NULL: zero
  float* Sf;             // NULL: not wanted
  int dk, dv;            // the problem's own (dq and dk exchange the call's)
  int s0_t;              // S0 is stored [d_v][d_k]
  int lag;
  int mode;
  float a, b, c;
  int mq, mk, mv;  // the tensors' maps in DecayArgs::map
};

// The tensor-core kernel's share of a call.  Every sequence, for every problem and head, is a unit of at least one
// chunk of 128 tokens; the chunks of all units in a row are dealt to the blocks in equal runs, so a block walks the end
// of a unit, whole units, and the beginning of one.  `gran` chunks are never parted (1, or all of a unit).
struct DecayDeal {
  int grid;     // blocks
  int gran;
  int chunks;   // of a unit (without cu)
  int nprob;
  // Whether one pass does it, the blocks handing states on: a block first makes known what its last unit's part in the run
  // adds to the state (walking that part for its state alone, unless it may be walked in full at once), and comes to the
  // end of its first unit, which needs the states of the blocks before it, last.  Blocks are numbered as they start, and
  // wait only for lower numbers, which wait for nothing before they hand on.
  int handoff;
  int joined;   // else: a first pass forms the states of the cut parts, and a kernel of their own joins them
};

// How the tensor-core kernel fetches tiles: token by token, or by TMA from whole-row or column maps.
enum { kFetchTokens = 0, kFetchRows = 1, kFetchCols = 2 };
constexpr int kColRun = 16;  // tokens of a column map's box

struct DecayArgs {
  alignas(64) CUtensorMap map[4];
  alignas(64) CUtensorMap omap[3];  // the problems' outputs
  int fetch;
  DecayProblem p[3];
  const float* g;  // [H] log decays
  const int* cu;
  const int* slots;
  int n_slots;
  int B, H, L, Hg, Wg;
  int seg;        // tokens of a segment
  int nps;        // segments of a sequence of L tokens (without cu)
  int states;     // segment states of a problem and head
  DecayDeal deal;
  uint32_t* flag;     // [block] a block's state has been handed over (left zero)
  uint32_t* counter;  // blocks started, blocks done (left zero)
  float* segst;   // tensor core: [2][block][D * D], what a block's cut unit adds to its state, and the copy of its S0; else [problem][segment][H][D * D] segment states
  long long segst_problem;  // elements between problems there
  uint32_t* status;
  // The tensor core's waits: whether a limit below the default holds, which has passed after some 0.1 ms, and the chunk of
  // a block whose loads are made to outlast it (-1: none).
  int short_wait, late_chunk;
};

struct DecayUnit {
  int b, i, nseg;  // sequence, segment of it, its segments
  int first, len;  // the sequence's first row and length
  int t0, n;       // the segment's first scan position and its tokens
  int slot;        // state of the sequence, -1: none
  int first_state; // the sequence's first segment among the segment states (those of several segments have any)
};

// Row of scan position t of unit u's sequence.
template <typename U>
__device__ __forceinline__ int decay_row(const DecayArgs& a, const U& u, int mode, int t) {
  if (a.cu) return u.first + ((mode & 1) ? u.len - 1 - t : t);
  return u.first + scan_to_grid(t, a.L, a.Hg, a.Wg, mode);
}

// Bounds of sequence b among the packed rows, forced into 0 .. L.
__device__ __forceinline__ void decay_bounds(const DecayArgs& a, int b, int& lo, int& hi) {
  lo = min(max(a.cu[b], 0), a.L);
  hi = min(max(a.cu[b + 1], lo), a.L);
}

// The state slot of sequence b, -1: none (reported where the caller asked for one); one warp.
__device__ __forceinline__ int decay_slot(const DecayArgs& a, int b) {
  if (!a.slots) return b;
  int slot = a.slots[b];
  bool bad = slot >= a.n_slots;
  for (int j = threadIdx.x & 31; j < b && slot >= 0; j += 32) bad |= a.slots[j] == slot;
  if (__any_sync(0xFFFFFFFFu, bad)) {
    slot = -1;
    if ((threadIdx.x & 31) == 0) set_status(a.status, DIG_ERR_INVALID_ARGUMENT);
  }
  return slot;
}

// The unit of segment slot `sidx` of the call; every lane of the calling warp
// gets it.  False: the call has fewer segments, or the unit's sequence reaches past
// the call's slots, one per block of gridDim.x, or past its segment states.  Only
// sequences that overlap, as those of descending offsets do, can: they come to more
// tokens than the rows that both are counted for, and are left out whole.
__device__ __forceinline__ bool decay_unit(const DecayArgs& a, int sidx, DecayUnit& u) {
  const int lane = threadIdx.x & 31;
  if (!a.cu) {
    u.b = sidx / a.nps;
    u.i = sidx - u.b * a.nps;
    u.nseg = a.nps;
    u.first = u.b * a.L;
    u.len = a.L;
    u.first_state = u.b * a.nps;
  } else {
    int base = 0, states = 0;
    bool found = false;
    for (int b0 = 0; b0 < a.B && !found; b0 += 32) {
      int lo = 0, hi = 0, ns = 0;
      if (b0 + lane < a.B) {
        decay_bounds(a, b0 + lane, lo, hi);
        ns = max(1, (hi - lo + a.seg - 1) / a.seg);
      }
      int inc = ns, st = ns > 1 ? ns : 0;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, inc, m), y = __shfl_up_sync(0xFFFFFFFFu, st, m);
        if (lane >= m) inc += x, st += y;
      }
      const unsigned has = __ballot_sync(0xFFFFFFFFu, base + inc > sidx);
      if (has) {
        const int src = __ffs(has) - 1;
        u.b = b0 + src;
        u.nseg = __shfl_sync(0xFFFFFFFFu, ns, src);
        u.i = sidx - base - (__shfl_sync(0xFFFFFFFFu, inc, src) - u.nseg);
        u.first = __shfl_sync(0xFFFFFFFFu, lo, src);
        u.len = __shfl_sync(0xFFFFFFFFu, hi, src) - u.first;
        u.first_state = states + __shfl_sync(0xFFFFFFFFu, st, src) - u.nseg;
        found = true;
      }
      base += __shfl_sync(0xFFFFFFFFu, inc, 31);
      states += __shfl_sync(0xFFFFFFFFu, st, 31);
    }
    if (!found || sidx - u.i + u.nseg > (int)gridDim.x || (u.nseg > 1 && u.first_state + u.nseg > a.states)) return false;
  }
  u.t0 = u.i * a.seg;
  u.n = min(a.seg, u.len - u.t0);
  u.slot = decay_slot(a, u.b);
  return true;
}

// Chunks of 128 tokens that a sequence of n tokens counts for (an empty one has a state to pass on).
__device__ __forceinline__ int deal_chunks(int n) { return n > 128 ? (n + 127) / 128 : 1; }

// Chunks of all sequences of a packed call (one warp).
__device__ __forceinline__ long long deal_total(const DecayArgs& a) {
  long long s = 0;
  for (int b = threadIdx.x & 31; b < a.B; b += 32) {
    int lo, hi;
    decay_bounds(a, b, lo, hi);
    s += deal_chunks(hi - lo);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
  return s;
}

// A block's walk through part of a unit.
struct DecayPiece {
  int b, h, z;           // sequence, head, problem
  int first, len;        // the sequence's first row and length
  int t0, n;             // the piece's first scan position and its tokens
  int chunks;            // of the piece
  int unit_chunks;       // of the unit
  bool last;             // whether the unit ends with it
  int slot;              // state of the sequence, -1: none
  long long unit_start;  // the unit's first chunk among all units'
};

// a / b, mostly of small numbers (a 64-bit division is a hundred instructions).
__host__ __device__ __forceinline__ long long deal_div(long long a, long long b) {
  return ((a | b) >> 31) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}
// `grains` dealt to `grid` blocks: the first `rem` of them take q + 1 each, the others q.
struct DealRuns {
  long long q;
  int rem;
  __host__ __device__ __forceinline__ DealRuns(long long grains, int grid) : q(deal_div(grains, grid)), rem((int)(grains - q * grid)) {}
  __device__ __forceinline__ long long start(int i) const { return i * q + min(i, rem); }
  __device__ __forceinline__ int block_of(long long x) const {
    const long long head = rem * (q + 1);
    return (int)(x < head ? deal_div(x, q + 1) : rem + deal_div(x - head, q));
  }
};

// The piece that starts at chunk r of all units', `per` of each (problem, head), and ends before chunk r1; one warp.
__device__ __forceinline__ void decay_piece(const DecayArgs& a, long long per, long long r, long long r1, DecayPiece& u) {
  const int lane = threadIdx.x & 31;
  const long long zh = deal_div(r, per);
  const long long w = r - zh * per;
  u.z = (int)deal_div(zh, a.H);
  u.h = (int)(zh - (long long)u.z * a.H);
  int nch, c0;
  if (!a.cu) {
    nch = a.deal.chunks;
    u.b = (int)deal_div(w, nch);
    c0 = (int)(w - (long long)u.b * nch);
    u.first = u.b * a.L;
    u.len = a.L;
  } else {
    long long base = 0;
    nch = 1, c0 = 0, u.b = 0, u.first = 0, u.len = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      int lo = 0, hi = 0, ns = 0;
      if (b0 + lane < a.B) {
        decay_bounds(a, b0 + lane, lo, hi);
        ns = deal_chunks(hi - lo);
      }
      int inc = ns;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, inc, m);
        if (lane >= m) inc += x;
      }
      const unsigned has = __ballot_sync(0xFFFFFFFFu, base + inc > w);
      if (has) {
        const int src = __ffs(has) - 1;
        u.b = b0 + src;
        nch = __shfl_sync(0xFFFFFFFFu, ns, src);
        c0 = (int)(w - (base + __shfl_sync(0xFFFFFFFFu, inc, src) - nch));
        u.first = __shfl_sync(0xFFFFFFFFu, lo, src);
        u.len = __shfl_sync(0xFFFFFFFFu, hi, src) - u.first;
        break;
      }
      base += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
  }
  u.chunks = (int)min((long long)(nch - c0), r1 - r);
  u.unit_chunks = nch;
  u.last = c0 + u.chunks == nch;
  u.t0 = 128 * c0;
  u.n = max(min(u.len - u.t0, 128 * u.chunks), 0);
  u.unit_start = r - c0;
  u.slot = decay_slot(a, u.b);
}

// Reports offsets that do not ascend within 0 .. L (one warp of the call does this).
__device__ __forceinline__ void decay_check_offsets(const DecayArgs& a) {
  for (int b = threadIdx.x & 31; b < a.B; b += 32)
    if (a.cu[b] < 0 || a.cu[b + 1] < a.cu[b] || a.cu[b + 1] > a.L) set_status(a.status, DIG_ERR_INVALID_ARGUMENT);
}

// lambda^i = hi + lo for a whole i >= 0, from the log decay as given (lambda^0 = 1 also for lambda = 0).
__device__ __forceinline__ float2 decay_pow(float g, long long i) {
  const double p = i == 0 ? 1.0 : exp(static_cast<double>(g) * static_cast<double>(i));
  const float hi = static_cast<float>(p);
  return make_float2(hi, isfinite(hi) ? static_cast<float>(p - hi) : 0.f);
}

// The launches of a call (FP32 pipes: two passes where a sequence may have several segments, `multi`).
cudaError_t launch_decay_f32(const DecayArgs& a, int nprob, int nseg_total, bool multi, int D, int dtype, int out_dtype,
                             cudaStream_t s);
cudaError_t launch_decay_tc(const DecayArgs& a, int D, cudaStream_t s);

}  // namespace dig
