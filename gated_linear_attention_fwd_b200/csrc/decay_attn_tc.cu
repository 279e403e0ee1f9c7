// decay_attn_tc.cu -- head-decay linear attention on the tensor core (bf16 inputs
// and outputs).
//
// One block walks its share of the (sequence, head) units in chunks of 128 tokens; per
// chunk (n tokens, entry state S, the problem's factors a, b, c):
//   P  = q k^T,            P[t][s] <- a lambda^(t-s) P[t][s] for s <= t, else 0
//   dS = khat^T v,         khat_s = b lambda^(n-1-s) k_s
//   O1 = q S,              O2 = P v,      o[t] = c lambda^(t+1) O1[t] + O2[t]
//   S  = lambda^n S + dS
// all four products by tcgen05.mma with fp32 accumulators in tensor memory.  One
// warp issues them; with TMA one fetches the tiles, one stores outputs and one plans,
// token by token three fetch a tile each and one of these plans too; the rest (4 warps
// per 32 lanes at D = 128, 2 at D = 64, so that a thread holds 32 columns of S, dS and O
// either way) do what is between the products:
//   - q, k, v tiles (raw bf16, exact) come two chunks deep (three in the first pass) into 128-byte-swizzled
//     tiles of 64 channels, by TMA (boxes of whole rows, or of runs of a grid
//     column; a reversed scan keeps its tiles in memory order and mirrors the mask)
//     or, where alignment or the grid does not allow that, token by token through
//     cp.async.  Rows past the segment and channels past the head are zero.  The same
//     bytes serve K-major (q k^T) and MN-major (v as the second operand);
//   - P is masked, scaled and split into two bf16 terms in place in tensor memory
//     and read from there as the first operand of P v.  The decays are applied to
//     the fp32 product (lambda^(t-s) itself, no quotient of powers: any lambda from
//     0 to 1 is in range);
//   - S lives in fp32 registers (one key channel per lane) and is left in shared
//     memory as one bf16 term, the second operand of q S: off by at most half a
//     bf16 step, as the output's own rounding is (at D = 128 a second term has no room
//     beside two chunks of tiles; fp32 outputs take the FP32 pipes, which do without).  lambda^n is applied as hi + lo and dS is summed apart
//     from S: a tensor-core accumulator that carried S through the sequence would
//     cut a little off it at every addition;
//   - khat^T (lane = channel) goes to tensor memory through transposing matrix
//     loads: two bf16 terms where the state only feeds outputs, three, exact to
//     fp32, where the final state itself is asked for and the chunk's part of it has
//     not decayed below 2^-10 by then (two terms leave 2^-17 of that).
// Products run in the order of their issue, which lets them share columns: O2 lies
// where dS stood, and khat (D = 128: its third term) where P and O1 come to stand.
// At D = 128 khat of the next chunk is formed while P v runs, and q k^T of the next
// chunk follows P v at once.  At D = 64 two blocks share an SM instead.
//
// The chunks of all sequences, heads and (backward) problems are dealt to the blocks
// in equal runs; a block walks its run piece by piece, the next piece planned by a
// warp of its own meanwhile.  decay_attn.h says how a sequence's state gets past the
// end of a run, decay_attn.cu what that costs.
//
// What bounds it (B200, SM clock about 1.75 GHz under load): at 128 x 128 a chunk
// takes 5700 to 6000 cycles, against 2950 ns x clock = 5200 that its 128 KB take at
// the SM's share of the measured copy rate and about 3100 of products; the issue
// slots are half used, and a chunk's chain (mask, dS, update, P v, output) does the
// rest.  A chunk whose state needs three terms takes 7800, one walked for its state
// alone 3000, a piece's start 4000, a block's 10000.  At 32 x 64 a chunk takes 8000 in
// each of two blocks: its chain.  Whole calls: 16382 packed tokens, 16 heads of
// 128/128, 112 to 119 us (2.5 TB/s); 2 x 12544 tokens, 6 heads of 32/64, 53 us; backward of
// 4 x 4096 tokens, 16 heads of 128/128, 217 to 229 us (2.2 TB/s).  Token by token 16384
// tokens of 16 heads of 36/72 take 211 us, their backward 608.
//
// Every wait on a barrier or a flag is bounded.  After one was given up the roles pass over
// what is left of the piece without leaving each other at its barriers, wait for the loads,
// stores and products in flight and leave together; the status says so, and flags and
// counters end at zero as ever.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "decay_attn.h"
#include "sm100.cuh"
#include "tma.cuh"

namespace dig {

namespace {

constexpr int C = 128;  // tokens of a chunk

// 16 consecutive columns of this thread's lane, loaded and waited for in one statement (no use can move above the wait).
__device__ __forceinline__ void tmem_take16(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
// The same from two places.
__device__ __forceinline__ void tmem_take16x2(uint32_t taddr, uint32_t taddr2, float* v, float* w) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]), "=f"(w[4]), "=f"(w[5]), "=f"(w[6]), "=f"(w[7]), "=f"(w[8]), "=f"(w[9]), "=f"(w[10]), "=f"(w[11]), "=f"(w[12]), "=f"(w[13]), "=f"(w[14]), "=f"(w[15])
      : "r"(taddr), "r"(taddr2)
      : "memory");
}
// 16 lanes x 16 columns: register 2 i (2 i + 1) of thread T is lane T / 4 (+ 8), column 4 i + T % 4, the
// arrangement in which transposing matrix loads leave a tile.
__device__ __forceinline__ void tmem_put_16x16(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Four 8 x 8 matrices of 16-bit values, each transposed: thread T gets row T / 4, values 2 (T % 4) and + 1 of each.
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// One row piece of 16 or 8 bytes; nothing is read and zeros are written where `bytes` is 0.
template <int N>
__device__ __forceinline__ void cp_piece(uint32_t dst, const void* src, int bytes) {
  if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// Barrier `id` over `n` threads; true for all of them if `x` is for any.
__device__ __forceinline__ bool bar_or(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 x;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(addr) : "memory");
  return x;
}
// Moves registers between the warps of a block (warpgroup-wide; the sums stay within the launch's total).
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t f2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void f2_out(uint64_t v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  float x, y;
  f2_out(v, x, y);
  return pack_bf16x2(x, y);
}
// The next bf16 term of a pair of values: packed, and taken off the values.
__device__ __forceinline__ uint32_t take_term(uint64_t& v) {
  const uint32_t t = pack2(v);
  v = fma2(f2(__uint_as_float(t << 16), __uint_as_float(t & 0xFFFF0000u)), f2(-1.f, -1.f), v);
  return t;
}

// The products and their commit, by the one thread of a warp whose `on` is set: the warp's control flow and operands
// stay uniform, so that the descriptors are formed in uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "setp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "setp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(on)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// The low half of the timer: waits end within its four seconds.
__device__ __forceinline__ uint32_t timer_ns() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
// What sh.abort holds: a wait was given up; the call's limit is a short one (a test's).
enum { kGone = 1, kShort = 2 };
__device__ __forceinline__ bool gone(const int* abort) { return (*reinterpret_cast<const volatile int*>(abort) & kGone) != 0; }
// After a first probe that failed: probes until the phase completes, another warp has given up, or the limit has passed
// (then gives up).  The flag and the timer are looked at once in 32 probes, each of which suspends the thread for up to
// 4 us: the warps that wait share their issue slots with those that work.  A short limit has passed with the first 32.  (The
// limit itself as an operand of these loops costs the workers registers: 16384 tokens of 16 heads of 36/72 226 us, so 211.)
__device__ __forceinline__ bool mbar_wait_or(uint64_t* bar, uint32_t parity, int* abort) {
  uint32_t t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(abort)) break;
    const uint32_t now = timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > (uint32_t)kSpinLimitNs) break;
  }
  *reinterpret_cast<volatile int*>(abort) = kGone | kShort;
  return false;
}

// Second operand read MN-major: rows are the contracted index, atoms of 64 columns `atom` bytes apart.
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr, uint32_t atom) {
  uint64_t d = sdesc_sw<128>(addr);
  d &= ~(static_cast<uint64_t>(0x3FFF) << 16);
  return d | static_cast<uint64_t>((atom >> 4) & 0x3FFF) << 16;
}

enum { kFull, kLast, kFullLag, kLastLag, kRun, kRun1, kSteps };

template <int D, bool STATES>
struct TcCfg {
  static constexpr bool SMALL = D == 64;
  static constexpr int CG = D / 32;               // threads per lane
  static constexpr int NT = 128 * CG;             // worker threads; 128 more issue and fetch
  static constexpr int ATOM = C * 128;            // bytes of 64 channels of a tile
  static constexpr int TILE = ATOM * (D / 64);
  static constexpr int PER = STATES ? 2 : 3;      // tiles of a chunk: k, v, q
  static constexpr int S_ATOM = D * 128;
  static constexpr int ST = STATES ? 3 : 2;       // chunks in shared memory
  static constexpr int OFF_S = PER * ST * TILE;
  static constexpr int OFF_T = OFF_S + (STATES ? 0 : S_ATOM * (D / 64));
  // Registers: 512 x 104 + 128 x 56 of 640 x 96 (D = 128), 256 x 96 + 128 x 48 of 384 x 80 (D = 64).  What does not fit goes
  // to local memory, for which little L1 is left beside the tiles: a load from there costs a trip to L2.
  static constexpr int WORKER_REGS = SMALL ? 96 : 104, SERVICE_REGS = SMALL ? 48 : 56;
  // tensor memory columns (khat: 64 a term)
  static constexpr int TM_COLS = SMALL ? 256 : 512;
  static constexpr int TM_P = 0, TM_O1 = 128, TM_DS = SMALL ? 192 : (STATES ? 384 : 256), TM_O2 = TM_DS;
  static constexpr int PW = C / CG;               // P columns of a thread
  static constexpr bool THREE_AT_ONCE = SMALL || STATES;
  // first column of term i of khat of chunk m
  __device__ static __forceinline__ uint32_t tm_k(int m, int i) {
    if (SMALL) return 64 * i;
    if (STATES) return (m & 1) * 192 + 64 * i;
    return i < 2 ? 384 + 64 * i : TM_O1;
  }
  // the same where only the state is formed, which leaves P and O1 free: two places
  __device__ static __forceinline__ uint32_t tm_k_state(int m, int i) {
    if (SMALL || STATES) return tm_k(m, i);
    return i < 2 ? (m & 1 ? 0 : 384) + 64 * i : TM_O1 + 64 * (m & 1);
  }
};

// A piece and what its chunks need of its head's decay.
struct TcPiece {
  float pw[C + 4];            // lambda^i
  float pa[32];               // a lambda^i
  alignas(16) float p16[16];  // lambda^(15-i), mirrored tiles: lambda^i
  float2 step[kSteps];        // lambda^i = hi + lo of a chunk's or a block's run of tokens
  DecayPiece u;
  float g;                    // the head's log decay
  int keep;                   // whether the unit's final state is asked for
  int j0;                     // the first block whose state is to be joined
  int rem;                    // the blocks before this one have the longer runs
  long long run;              // chunks of the shorter runs
  int state;                  // only the state is formed
  int publish;                // the state at its end is handed on
  int more;                   // 0: there is no such piece
};

template <int ST>
struct TcTables {
  TcPiece piece[2];
  float wk[ST][C];                  // b lambda^(n-1-s) of chunk m in m % ST, 0 past its end
  uint64_t full[3][ST];             // tile x (k, v, q) of the chunk has come
  uint64_t landed[2];               // k and v of a chunk that ends inside its tiles
  uint64_t free_[3][ST];            // tile x (k, v, q) of the chunk is no longer read
  uint64_t bar_k, bar_p;            // the workers': khat (with S) written, P written (and dS read)
  uint64_t bar_qk, bar_ds, bar_qs, bar_pv, bar_end;  // the tensor core's
  uint64_t bar_out[2];              // the outputs of chunk m are staged, m & 1
  // how the chunks are dealt, and what of this block's run is left
  long long per, at, end;
  struct {
    long long at, end;
    int state, publish;
  } todo[4];                        // what of the run comes after that, in order
  int next;
  int me;                           // this block's number
  uint32_t tmem;
  int abort;
};

// A block's walk through its run, piece by piece; STATES: only what its cut unit adds to its state (the first of two passes).
// FETCH: how tiles come (one way a kernel: what an SM has to hold of its code counts).
template <int D, bool STATES, int FETCH>
__global__ void __launch_bounds__(TcCfg<D, STATES>::NT + 128, D == 64 ? 2 : 1) decay_tc_kernel(const __grid_constant__ DecayArgs a) {
  using F = TcCfg<D, STATES>;
  static_assert(F::OFF_T + sizeof(TcTables<F::ST>) <= (D == 64 ? 113 : 227) * 1024, "the blocks of an SM fit its shared memory");
  constexpr int NT = F::NT, CG = F::CG, W0 = NT / 32;
  extern __shared__ __align__(1024) uint8_t smem[];
  using Tables = TcTables<F::ST>;
  Tables& sh = *reinterpret_cast<Tables*>(smem + F::OFF_T);
  const int tid = threadIdx.x, warp = tid >> 5, ln = tid & 31;
  const uint32_t sb = smem_u32(smem);
  if (warp == W0) {
    tmem_alloc(&sh.tmem, F::TM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < F::ST; ++i) {
      for (int x = 0; x < 3; ++x) {
        mbar_init(&sh.full[x][i], 1);
        mbar_init(&sh.free_[x][i], x == 1 && !STATES && FETCH == kFetchTokens ? NT / 32 : 1);
      }
    }
    mbar_init(&sh.bar_out[0], NT / 32);
    mbar_init(&sh.bar_out[1], NT / 32);
    mbar_init(&sh.bar_k, NT / 32);
    mbar_init(&sh.bar_p, NT / 32);
    mbar_init(&sh.bar_qk, 1);
    mbar_init(&sh.bar_ds, 1);
    mbar_init(&sh.bar_qs, 1);
    mbar_init(&sh.bar_pv, 1);
    mbar_init(&sh.bar_end, 1);
    mbar_init(&sh.landed[0], 1);
    mbar_init(&sh.landed[1], 1);
    sh.abort = a.short_wait ? kShort : 0;
    fence_mbar_init();
  }
  // After a first pass (which started after everything before this call had ended) a block plans, fetches its first tiles
  // and waits for that pass only before it touches states.
  const bool early = !STATES && FETCH != kFetchTokens && a.deal.joined;
  auto depend = [&]() {
    griddep_wait();
    griddep_launch_dependents();
  };
  if (FETCH != kFetchTokens && warp == W0 + 1 && (ln < 4 ? ln < 3 || a.deal.nprob > 1 : ln - 4 < a.deal.nprob))
    asm volatile("prefetch.tensormap [%0];" ::"l"(tmap_addr(ln < 4 ? a.map[ln] : a.omap[ln - 4])) : "memory");
  const bool on = (sb & 1023u) == 0;  // the swizzled tiles start at 1024-byte boundaries
  // Waits are bounded by the call's limit; after one gave up every other one does, nothing more is issued and the block leaves.
  bool timed_out = false;
  auto wait_bar = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    if (!timed_out && !mbar_wait_or(bar, parity, &sh.abort)) timed_out = true;
    return !timed_out;
  };

  // Where the first piece follows from the arguments alone, it is planned while the kernels before this one end.
  const bool planned = !a.cu && !a.slots && !a.deal.handoff;
  // Every role walks the pieces, parted by block-wide barriers; one warp plans the next while this one is walked.
  auto plan = [&](int k) {
    TcPiece& t = sh.piece[k & 1];
    long long per;
    if (k == 0) per = a.cu ? deal_total(a) : (long long)a.B * a.deal.chunks;
    else per = sh.per;
    const long long grains = deal_div(per * a.H * a.deal.nprob, a.deal.gran);
    const int grid = (int)min((long long)a.deal.grid, grains);
    const DealRuns runs(grains, grid);
    long long r = 0, r1 = 0;  // what comes next
    int me = blockIdx.x, state = 0, publish = 0;
    if (k == 0) {
      if (a.deal.handoff) {
        if (ln == 0) me = (int)atomicAdd(a.counter, 1u);
        me = __shfl_sync(0xFFFFFFFFu, me, 0);
      }
      if (on && me < grid) {
        r = runs.start(me) * a.deal.gran;
        r1 = runs.start(me + 1) * a.deal.gran;
      }
      if (ln == 0) sh.next = 4;
      if (a.deal.handoff && r < r1) {
        DecayPiece u;
        decay_piece(a, per, r, r1, u);  // the run's first unit: what is left of it, unless the run starts with it
        const long long head = u.unit_start < r ? min(u.unit_start + u.unit_chunks, r1) : r;
        decay_piece(a, per, r1 - 1, r1, u);  // and its last: what the run has of it, unless it ends there
        const bool open = !u.last;
        const long long tail = open ? max(r, u.unit_start) : r1;
        // walked in full at once where it begins with the unit and the next block ends that, after other work as long
        const long long end = u.unit_start + u.unit_chunks, next_end = runs.start(min(me + 2, grid));
        const bool once = u.unit_start >= r && end <= next_end && r1 - tail <= next_end - end + 2;
        if (ln == 0) {
          int i = 4;
          auto put = [&](long long at, long long end, int st, int pub) {
            if (at < end) {
              --i;
              sh.todo[i].at = at, sh.todo[i].end = end, sh.todo[i].state = st, sh.todo[i].publish = pub;
            }
          };
          const bool middle = open && u.unit_start < r;  // the run is a part of one unit
          if (!middle) put(r, head, 0, 0);
          if (open && !once) put(tail, r1, 0, 0);
          if (!middle) put(head, tail, 0, 0);
          if (open) put(tail, r1, !once, 1);
          sh.next = i;
        }
        r = r1 = 0;
      }
    } else {
      me = sh.me;
      r = sh.at;
      r1 = sh.end;
    }
    __syncwarp();
    int next = sh.next;
    if (r >= r1 && next < 4) {
      r = sh.todo[next].at;
      r1 = sh.todo[next].end;
      state = sh.todo[next].state;
      publish = sh.todo[next].publish;
      ++next;
    }
    __syncwarp();
    bool more = r < r1;
    if (more) {
      DecayPiece u;
      if (STATES) {  // the last unit's, if it goes on in the next block
        decay_piece(a, per, r1 - 1, r1, u);
        r = max(r, u.unit_start);
      }
      decay_piece(a, per, r, r1, u);
      if (STATES) more = !u.last;
      if (ln == 0) {
        t.u = u;
        if (k > 0 || !planned) t.g = a.g[u.h];
        t.keep = a.p[u.z].Sf && u.slot >= 0;
        t.j0 = a.deal.joined ? me - 1 : runs.block_of(u.unit_start);
        t.state = state;
        t.publish = publish;
        t.rem = runs.rem;
        t.run = runs.q;
      }
      if (k > 0 && more && u.t0 == 0 && (u.last || publish) && a.p[u.z].S0 && u.slot >= 0) {  // on the way to L2 by the time the piece starts
        const DecayProblem& p = a.p[u.z];
        const char* s0 = reinterpret_cast<const char*>(p.S0 + ((size_t)u.slot * a.H + u.h) * p.dk * p.dv);
        for (int i = 128 * ln; i < 4 * p.dk * p.dv; i += 128 * 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(s0 + i));
      }
      r = STATES ? r1 : r + u.chunks;
    }
    if (ln == 0) {
      t.more = more;
      sh.per = per;
      sh.at = r;
      sh.end = r1;
      sh.next = next;
      sh.me = me;
    }
    __syncwarp();
  };
  // The powers of a piece, by `step` threads.
  auto powers = [&](TcPiece& t, int first, int step) {
    if (!t.more) return;
    const DecayProblem& p = a.p[t.u.z];
    const bool rev = FETCH != kFetchTokens && (p.mode & 1);
#pragma unroll 1
    for (int j = first; j < C + kSteps; j += step) {
      // from C on: lambda to the tokens of a whole chunk, of the last one, of either where its first token counts
      // without its decay (lag), and of the shorter and the longer of the blocks' runs
      const int last = t.u.n - max(t.u.n - 1, 0) / C * C;
      const long long i = j <= C             ? j
                          : j == C + kLast    ? last
                          : j == C + kFullLag ? C - 1
                          : j == C + kLastLag ? max(last - 1, 0)
                                              : (t.run + (j - C - kRun)) * C;
      const float2 w = decay_pow(t.g, i);
      if (j <= C) t.pw[j] = w.x;
      if (j >= C) t.step[j - C] = w;
      if (j < 16) t.p16[rev ? j : 15 - j] = w.x;
      if (j < 32) t.pa[j] = p.a * w.x;
    }
  };
  if (!early && !planned) depend();
  if (warp == W0 + 3) plan(0);
  if (!early && planned) depend();
  if (!on && tid == 0) set_status(a.status, DIG_ERR_CUDA);
  if (!STATES && a.cu && blockIdx.x == 0 && warp == 0) decay_check_offsets(a);
  if (planned && warp == W0 + 3 && ln == 0 && sh.piece[0].more) sh.piece[0].g = a.g[sh.piece[0].u.h];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  if (tid < NT) powers(sh.piece[0], tid, NT);
  __syncthreads();
  // Every role is through with the piece; false: one gave up.  The second barrier keeps the others from the next piece's
  // waits until all have read the flag: put up by one of those, it would part roles that have read it from those that have not.
  auto piece_done = [&]() {
    named_bar(0, NT + 128);
    const bool leave = gone(&sh.abort);
    named_bar(0, NT + 128);
    return !leave;
  };
  auto tile = [&](int x, int m) { return sb + ((m % F::ST) * F::PER + x) * F::TILE; };  // x: 0 k, 1 v, 2 q
  // a value that every lane has, as one the compiler knows to be the same in all of them
  auto same = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
  // bf16 terms of khat in the chunk from which on `left` tokens of the piece are left (0: nothing needs the state after it)
  auto terms_of = [&](const TcPiece& t, int left) {
    const int after = t.u.len - t.u.t0 - t.u.n + left - C;  // tokens of the sequence after the chunk
    const bool needed = STATES || left > C || t.publish || (t.u.last && t.keep);
    return same(!needed ? 0 : t.keep && t.g * max(after, 0) >= -7.f ? 3 : 2);
  };
  // Waits, as long as wait_bar would, for another block's flag.
  auto wait_flag = [&](const uint32_t* f) {
    uint32_t t0 = 0;
    while (true) {
      uint32_t v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(f) : "memory");
      if (v || timed_out || gone(&sh.abort)) return;
      const uint32_t now = timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > (a.short_wait ? 100000u : (uint32_t)kSpinLimitNs)) {
        timed_out = true;
        sh.abort = kGone | kShort;
      }
    }
  };
  int base = 0;  // chunks before this piece: they are counted through the pieces

  if (warp == W0) {
    // ---- the issuing warp
    regs_down<F::SERVICE_REGS>();
    if (early) depend();
    const uint32_t one = elect_one();
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
#pragma unroll 1
    for (int piece = 0; sh.piece[piece & 1].more; ++piece) {
    const TcPiece& tab = sh.piece[piece & 1];
    const DecayPiece& u = tab.u;
    const DecayProblem& p = a.p[same(u.z)];
    const int end = base + same((u.n + C - 1) / C);
    const int kk = (p.dk + 15) / 16;       // K-steps over the key channels
    const int nv = (p.dv + 15) / 16 * 16;  // columns of the products with v or S
    int left = same(u.n);                  // tokens from the current chunk on
    const uint32_t id_qk = idesc_bf16(128, 128), id_v = idesc_bf16(128, nv, false, true);
    const uint64_t s_desc = mn_desc(sb + F::OFF_S, F::S_ATOM);
    auto kstep = [](int ks) { return (uint64_t)(((ks >> 2) * F::ATOM + (ks & 3) * 32) >> 4); };
    auto qk = [&](int m) {
      const uint64_t kd = sdesc_sw<128>(tile(0, m)), qd = sdesc_sw<128>(tile(2, m));
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        if (ks < kk) mma_ss(one, tm + F::TM_P, qd + kstep(ks), kd + kstep(ks), id_qk, ks ? 1u : 0u);
      commit(one, &sh.bar_qk);
    };
    constexpr bool AHEAD = !STATES && !F::SMALL;  // q k^T of a chunk follows P v of the one before
    auto ready = [&](int x, int m) { return __all_sync(0xFFFFFFFFu, wait_bar(&sh.full[x][m % F::ST], (m / F::ST) & 1)); };
    const bool state = !STATES && same(tab.state);
    if (AHEAD && end > base && ready(0, base) && ready(2, base)) {
      if (state) commit(one, &sh.bar_qk);
      else qk(base);
    }
#pragma unroll 1
    for (int m = base; m < end; ++m, left -= C) {
      const uint32_t ph = m & 1;
      const int terms = terms_of(tab, left);
      if (!ready(1, m) || !__all_sync(0xFFFFFFFFu, wait_bar(&sh.bar_k, ph))) break;
      tc_fence_after();
      const uint64_t v0 = mn_desc(tile(1, m), F::ATOM);
#pragma unroll 1
      for (int i = terms - 1; i >= 0; --i) {  // the smallest terms first
        const uint32_t ka = tm + (state ? F::tm_k_state(m, i) : F::tm_k(m, i));
#pragma unroll
        for (int ks = 0; ks < C / 16; ++ks)
          mma_ts(one, tm + F::TM_DS, ka + 8 * ks, v0 + (uint64_t)((2048 * ks) >> 4), id_v, ks == 0 && i == terms - 1 ? 0u : 1u);
      }
      commit(one, &sh.bar_ds);
      if (STATES) {
        commit(one, &sh.free_[0][m % F::ST]);
        commit(one, &sh.free_[1][m % F::ST]);
      } else {
        if (F::SMALL) {
          if (!ready(2, m)) break;
          if (state) commit(one, &sh.bar_qk);
          else qk(m);
        }
        commit(one, &sh.free_[0][m % F::ST]);
        const uint64_t qd = sdesc_sw<128>(tile(2, m));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          if (ks < kk && !state) mma_ss(one, tm + F::TM_O1, qd + kstep(ks), s_desc + (uint64_t)((2048 * ks) >> 4), id_v, ks ? 1u : 0u);
        commit(one, &sh.bar_qs);
        commit(one, &sh.free_[2][m % F::ST]);
        if (!__all_sync(0xFFFFFFFFu, wait_bar(&sh.bar_p, ph))) break;
        tc_fence_after();
        if (!state)
#pragma unroll
        for (int i = 1; i >= 0; --i)  // a K-step's 16 columns: 8 of the first term, 8 of the second
#pragma unroll
          for (int ks = 0; ks < C / 16; ++ks)
            mma_ts(one, tm + F::TM_O2, tm + F::TM_P + 16 * ks + 8 * i, v0 + (uint64_t)((2048 * ks) >> 4), id_v, i == 1 && ks == 0 ? 0u : 1u);
        commit(one, &sh.bar_pv);
        if (AHEAD && m + 1 < end) {
          if (!ready(0, m + 1) || !ready(2, m + 1)) break;
          if (state) commit(one, &sh.bar_qk);
          else qk(m + 1);
        }
      }
    }
    base = end;
    if (!piece_done()) break;
    }
    commit(one, &sh.bar_end);  // no product outlives the block
    mbar_wait(&sh.bar_end, 0, kSpinLimitNs);
  } else if (warp > W0) {
    // ---- the fetching warps
    regs_down<F::SERVICE_REGS>();
    uint32_t cleaned = 0;  // pieces whose last tiles were cleaned
    bool due = early;      // to wait for the first pass: the fetching warp first asks for two chunks
    if (early && warp != W0 + 1) depend();
#pragma unroll 1
    for (int piece = 0; sh.piece[piece & 1].more; ++piece) {
    const TcPiece& tab = sh.piece[piece & 1];
    const DecayPiece& u = tab.u;
    const DecayProblem& p = a.p[same(u.z)];
    const int h = same(u.h), end = base + same((u.n + C - 1) / C);
    const bool rev = FETCH != kFetchTokens && (p.mode & 1);
    if (warp == W0 + 3) {
      plan(piece + 1);
      powers(sh.piece[(piece + 1) & 1], ln, 32);
      __syncwarp();
    }
    // the weights of khat in chunk m of n tokens
    auto weights = [&](int m, int n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int s = rev ? C - 1 - 32 * i - ln : 32 * i + ln;
        sh.wk[m % F::ST][32 * i + ln] = s < n ? p.b * tab.pw[n - 1 - s] : 0.f;
      }
      __syncwarp();
    };
    // The place of tile x of chunk m is free; nothing more is fetched once a wait was given up (the others' signals need
    // not mean what they say then).
    auto freed = [&](int x, int m) {
      return m < F::ST || __all_sync(0xFFFFFFFFu, wait_bar(&sh.free_[x][m % F::ST], (m / F::ST - 1) & 1) &&
                                                      (FETCH == kFetchTokens || !gone(&sh.abort)));
    };
    // A test's: the v tile of this chunk of a block comes only after the others have given up (or a millisecond).
    auto late = [&](int m) {
      if (m != a.late_chunk) return;
      for (const uint32_t t0 = timer_ns(); !gone(&sh.abort) && timer_ns() - t0 < 1000000u;) {}
    };
    int asked = F::PER * end;  // tiles asked for by the piece's end, F::PER a chunk: k, q, v
    bool unclean = false;      // the last of those chunks is yet to be cleaned
    if constexpr (FETCH != kFetchTokens) {
      // one warp asks for a chunk's tiles in the order in which their places become free, one stores outputs, one plans
      if (warp == W0 + 1) {
        auto fetch = [&](int x, int m, bool clean) {
          const uint32_t dst = tile(x, m);
          const CUtensorMap& map = a.map[x == 0 ? p.mk : (x == 1 ? p.mv : p.mq)];
          uint64_t* bar = clean ? &sh.landed[x] : &sh.full[x][m % F::ST];
          const int atoms = min(D / 64, ((x == 1 ? p.dv : p.dk) + 63) / 64);
          if (ln == 0) {
            mbar_arrive_expect_tx(bar, atoms * F::ATOM);
            const int t0 = u.t0 + (m - base) * C;
            if constexpr (FETCH == kFetchRows) {
              const int r = (rev ? u.len - t0 - C : t0) + (a.cu ? u.first : 0);
              for (int i = 0; i < atoms; ++i) tma_load_5d(dst + i * F::ATOM, map, 64 * i, h, r, a.cu ? 0 : u.b, 0, bar);
            } else {
              const int f0 = rev ? a.L - t0 - C : t0;  // a multiple of the run, as L and the chunks are
              int col = f0 >= 0 ? f0 / a.Hg : 0, y = f0 >= 0 ? f0 - col * a.Hg : f0;
              for (int r = 0; r < C; r += kColRun) {
                const int yy = y < 0 ? a.Hg : y;  // before the first token: off the grid, zeros
                for (int i = 0; i < atoms; ++i) tma_load_5d(dst + i * F::ATOM + r * 128, map, 64 * i, h, yy, col, u.b, bar);
                y += kColRun;
                if (y >= a.Hg) y = 0, ++col;
              }
            }
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int m = base; m < end; ++m) {
          const int n = min(C, u.n - (m - base) * C);
          // packed: rows past the sequence's end are another's, and 0 times them need not be 0
          const bool clean = a.cu && n < C;
          if (due && m == 2) depend(), due = false;
          if (!freed(0, m)) {
            asked = F::PER * m;
            break;
          }
          weights(m, n);
          fetch(0, m, clean);
          if (!STATES) {
            if (!freed(2, m)) {
              asked = F::PER * m + 1, unclean = clean;
              break;
            }
            if (!tab.state) fetch(2, m, false);
            else if (ln == 0) mbar_arrive(&sh.full[2][m % F::ST]);  // nothing reads q
          }
          if (!freed(1, m)) {
            asked = F::PER * m + F::PER - 1, unclean = clean;
            break;
          }
          late(m);
          fetch(1, m, clean);
          if (clean) {
            bool ok = true;
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              ok = __all_sync(0xFFFFFFFFu, ok && wait_bar(&sh.landed[x], cleaned & 1));
              if (!ok) break;
              const int r0 = rev ? 0 : n, atoms = min(D / 64, ((x == 1 ? p.dv : p.dk) + 63) / 64);
#pragma unroll 1
              for (int i = ln; i < (C - n) * 8; i += 32)
                for (int j = 0; j < atoms; ++j) sts128(tile(x, m) + j * F::ATOM + (r0 + i / 8) * 128 + (i % 8) * 16, 0, 0, 0, 0);
              fence_async_smem();
              __syncwarp();
              if (ln == 0) mbar_arrive(&sh.full[x][m % F::ST]);
            }
            if (!ok) {
              asked = F::PER * (m + 1), unclean = true;
              break;
            }
            ++cleaned;
          }
        }
      }
      if (!STATES && warp == W0 + 2) {
        // whole chunks' outputs, from where the workers staged them (over the v tile, in its layout)
        const CUtensorMap& map = a.omap[same(u.z)];
        const int atoms = (p.dv + 63) / 64;
#pragma unroll 1
        for (int m = base; m < end; ++m) {
          if (!__all_sync(0xFFFFFFFFu, wait_bar(&sh.bar_out[m & 1], (m >> 1) & 1) &&
                                           !gone(&sh.abort))) break;
          const int t0 = u.t0 + (m - base) * C;
          if (ln == 0) {
            if (u.n - (m - base) * C >= C && !tab.state) {
              const uint32_t src = tile(1, m);
              if constexpr (FETCH == kFetchRows) {
                const int r = (rev ? u.len - t0 - C : t0) + (a.cu ? u.first : 0);
                for (int i = 0; i < atoms; ++i) tma_store_5d(map, 64 * i, h, r, a.cu ? 0 : u.b, 0, src + i * F::ATOM);
              } else {
                const int f0 = rev ? a.L - t0 - C : t0;
                int col = f0 / a.Hg, y = f0 - col * a.Hg;
                for (int r = 0; r < C; r += kColRun) {
                  for (int i = 0; i < atoms; ++i) tma_store_5d(map, 64 * i, h, y, col, u.b, src + i * F::ATOM + r * 128);
                  y += kColRun;
                  if (y >= a.Hg) y = 0, ++col;
                }
              }
              bulk_commit();
              bulk_wait_read_all();
            }
            mbar_arrive(&sh.free_[1][m % F::ST]);
          }
          __syncwarp();
        }
      }
    } else {
      // a warp per tile, in 16-byte pieces where all strides allow it, else in 8-byte ones
      const int x = warp - W0 - 1;
      if (x < F::PER) {
        const bool wide = (p.dk | p.dv) % 8 == 0 && (p.qs | p.ks | p.vs) % 8 == 0 &&
                          ((reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v)) & 15) == 0;
        const int d = x == 1 ? p.dv : p.dk;
        const long long st = 2 * (x == 0 ? p.ks : (x == 1 ? p.vs : p.qs));
        const char* src0 = static_cast<const char*>(x == 0 ? p.k : (x == 1 ? p.v : p.q)) + (size_t)h * d * 2;
#pragma unroll 1
        for (int m = base; m < end; ++m) {
          if (!freed(x, m)) break;
          if (x == 2 && !STATES && tab.state) {  // nothing reads q
            if (ln == 0) mbar_arrive(&sh.full[2][m % F::ST]);
            continue;
          }
          if (x == 1) late(m);
          const uint32_t dst = tile(x, m);
          if (x == 0) weights(m, min(C, u.n - (m - base) * C));
          int row[4];  // of tokens ln, ln + 32, ..
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int s = (m - base) * C + 32 * i + ln;
            row[i] = s < u.n ? decay_row(a, u, p.mode, u.t0 + s) : -1;
          }
          auto go = [&](auto bytes) {
            constexpr int N = decltype(bytes)::value;
            const int pieces = (d + 15) / 16 * 32 / N;  // of a row: the columns that a product reads
            const int inv = (65536 + pieces - 1) / pieces;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll 4
              for (int at = ln; at < 32 * pieces; at += 32) {
                const int r = (at * inv) >> 16, c = (at - r * pieces) * (N / 2), rr = 32 * i + r;
                const int gr = __shfl_sync(0xFFFFFFFFu, row[i], r);
                const bool ok = c < d && gr >= 0;
                const uint32_t to = dst + (c >> 6) * F::ATOM + rr * 128 + ((((c & 63) >> 3) ^ (rr & 7)) << 4) + (N == 16 ? 0 : (c & 4) * 2);
                cp_piece<N>(to, ok ? src0 + gr * st + 2 * c : src0, ok ? N : 0);
              }
          };
          if (wide) go(std::integral_constant<int, 16>{});
          else go(std::integral_constant<int, 8>{});
          cp_commit();
          cp_wait<0>();
          fence_async_smem();
          __syncwarp();
          if (ln == 0) mbar_arrive(&sh.full[x][m % F::ST]);
        }
      }
    }
    base = end;
    if (!piece_done()) {
      // No load outlives the block: the last one into each place (all of them, were it not for the giving up, are waited for
      // by the warps that read them).
      if (FETCH != kFetchTokens && warp == W0 + 1) {
#pragma unroll 1
        for (int i = max(asked - F::PER * F::ST, 0); i < asked; ++i) {
          const int m = i / F::PER, x = i % F::PER == 0 ? 0 : (i % F::PER == F::PER - 1 ? 1 : 2);
          const bool landed = unclean && m == (asked - 1) / F::PER && x < 2;
          mbar_wait(landed ? &sh.landed[x] : &sh.full[x][m % F::ST], (landed ? cleaned : m / F::ST) & 1, kSpinLimitNs);
        }
      }
      break;
    }
    }
    if (!STATES && FETCH != kFetchTokens && warp == W0 + 2) bulk_wait_all();  // nor does a store
  } else {
    // ---- the workers
    regs_up<F::WORKER_REGS>();
    const int t = tid & 127, cg = tid >> 7;  // token row or key channel (the thread's TMEM lane); column group
    const uint32_t lane = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    auto arrive = [&](uint64_t* bar) {       // the warp's writes to tensor and shared memory are done
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (ln == 0) mbar_arrive(bar);
    };

#pragma unroll 1
    for (int piece = 0; sh.piece[piece & 1].more; ++piece) {
    const TcPiece& tab = sh.piece[piece & 1];
    const DecayPiece& u = tab.u;
    const DecayProblem& p = a.p[same(u.z)];
    const int h = same(u.h);
    // tile row i holds scan position i of the chunk, or 127 - i where a reversed scan's tiles stay in memory order
    if (early && piece == 0) depend();
    const bool rev = FETCH != kFetchTokens && (p.mode & 1);
    const int kk = (p.dk + 15) / 16;                // K-steps over the key channels
    const int nv = (p.dv + 15) / 16 * 16;           // columns of the products with v or S
    const bool key = t < D && t < p.dk;             // this lane holds a key channel of the state
    // ---- the state the piece starts from: lane t = key channel, value channels 32 cg ..
    const bool state = !STATES && same(tab.state);
    if (!STATES && a.deal.handoff && u.t0 > 0 && !state) {  // the states of the blocks before
      for (int i = tab.j0 + ln; i < sh.me; i += 32) wait_flag(a.flag + i);
      __syncwarp();
    }
    float S[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) S[j] = 0.f;
    // S0 and S_final pass through 2 KB of S's shared memory a warp, half of its columns at a time, to 64-byte pieces of rows
    const uint32_t stage = sb + F::OFF_S + (cg * (D / 32) + (warp & 3)) * 2048;
    auto state_at = [&](auto* s0, int row, int half) {
      return reinterpret_cast<std::conditional_t<std::is_const_v<std::remove_pointer_t<decltype(s0)>>, const float4*, float4*>>(
          s0 + (size_t)(32 * (warp & 3) + row) * p.dv + 32 * cg + 16 * half + 4 * (ln & 3));
    };
    auto state_in = [&](int row, int half) { return 32 * (warp & 3) + row < p.dk && 32 * cg + 16 * half + 4 * (ln & 3) < p.dv; };
    // element (c, j) of a block's state: four value channels of consecutive key channels side by side
    auto block_state = [&](int i) { return reinterpret_cast<float4*>(a.segst + (size_t)i * (D * D)) + (cg * 8) * D + t; };
    if (t < D) {
      if (u.t0 == 0 && (STATES || u.last || tab.publish)) {
        if (p.S0 && u.slot >= 0) {
          const float* s0 = p.S0 + ((size_t)u.slot * a.H + h) * p.dk * p.dv;
          if (p.s0_t) {
            if (key) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (cg * 32 + j < p.dv) S[j] = s0[(size_t)(cg * 32 + j) * p.dk + t];
            }
          } else if constexpr (STATES) {  // (no shared memory to pass them through)
            if (key) {
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                if (cg * 32 + j < p.dv) {
                  const float4 x = *reinterpret_cast<const float4*>(s0 + (size_t)t * p.dv + cg * 32 + j);
                  S[j] = x.x, S[j + 1] = x.y, S[j + 2] = x.z, S[j + 3] = x.w;
                }
            }
          } else {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float4 x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = state_in(8 * i + ln / 4, half) ? __ldcg(state_at(s0, 8 * i + ln / 4, half)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                sts128(stage + swz_off<64>(8 * i + ln / 4, ln & 3), __float_as_uint(x[i].x), __float_as_uint(x[i].y), __float_as_uint(x[i].z), __float_as_uint(x[i].w));
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint4 v = lds128(stage + swz_off<64>(ln, i));
                const int j = 16 * half + 4 * i;
                S[j] = __uint_as_float(v.x), S[j + 1] = __uint_as_float(v.y), S[j + 2] = __uint_as_float(v.z), S[j + 3] = __uint_as_float(v.w);
              }
              __syncwarp();
            }
          }
        }
        if (STATES || state) {  // a copy for the walk in full, when the unit's last block may already have written S_final there
          float4* s0 = block_state(a.deal.grid + sh.me);
#pragma unroll
          for (int j = 0; j < 32; j += 4) s0[(j / 4) * D] = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
        }
      } else if (!STATES && !state) {
        // the states of the blocks that have walked the unit so far; at its start, the copy of S0
        const int j0 = u.t0 > 0 ? tab.j0 : a.deal.grid + sh.me, j1 = u.t0 > 0 ? sh.me : j0 + 1;
#pragma unroll 2
        for (int i = j0; i < j1; ++i) {
          const float4* ls = block_state(i);
          const float2 w = tab.step[i < tab.rem ? kRun1 : kRun];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 x = __ldcg(ls + (j / 4) * D);
            S[j] = fmaf(w.x, S[j], fmaf(w.y, S[j], x.x));
            S[j + 1] = fmaf(w.x, S[j + 1], fmaf(w.y, S[j + 1], x.y));
            S[j + 2] = fmaf(w.x, S[j + 2], fmaf(w.y, S[j + 2], x.z));
            S[j + 3] = fmaf(w.x, S[j + 3], fmaf(w.y, S[j + 3], x.w));
          }
        }
      }
    }
    int left = same(u.n);  // tokens from the current chunk on
    // S in bf16, rows = key channels (64 value channels each), the second operand of q S
    auto put_state = [&]() {
      if (t < D) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          const int jj = cg * 32 + j;
          sts128(sb + F::OFF_S + (jj >> 6) * F::S_ATOM + swz_off<128>(t, (jj & 63) >> 3), pack_bf16x2(S[j], S[j + 1]),
                 pack_bf16x2(S[j + 2], S[j + 3]), pack_bf16x2(S[j + 4], S[j + 5]), pack_bf16x2(S[j + 6], S[j + 7]));
        }
      }
    };
    if constexpr (!STATES) {
      named_bar(9, NT);  // S0 came through the same memory
      if (left > 0 && !state) put_state();
    }
    // khat^T of chunk m -> tensor memory: the warp's 32 channels, its group's tokens.  LAST: the last of three terms alone,
    // formed again once its place is free (held in registers meanwhile it would push others out to local memory).
    auto convert_k = [&](int m, int terms, auto last) {
      constexpr bool LAST = decltype(last)::value;
      if (terms == 0) return;
      const bool at_once = F::THREE_AT_ONCE || state;
      auto col = [&](int i) { return state ? F::tm_k_state(m, i) : F::tm_k(m, i); };
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int c = 32 * (warp & 3) + 16 * half;
        if (c >= 16 * kk) break;
        const uint32_t kt = tile(0, m) + (c >> 6) * F::ATOM;
        const int ch = ((c & 63) >> 3) + ((ln >> 3) & 1);
#pragma unroll 1
        for (int s0 = cg * F::PW; s0 < (cg + 1) * F::PW; s0 += 32) {
          uint32_t r[8];
          uint64_t x[8];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int tok = s0 + 16 * i + ((ln >> 4) << 3) + (ln & 7);
            ldsm_t(kt + tok * 128 + ((ch ^ (tok & 7)) << 4), r + 4 * i);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint64_t w = *reinterpret_cast<const uint64_t*>(&sh.wk[m % F::ST][s0 + 8 * (i >> 1) + 2 * (ln & 3)]);
            x[i] = mul2(f2(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xFFFF0000u)), w);
          }
          const uint32_t at = tmem + (static_cast<uint32_t>(c) << 16) + s0 / 2;
#pragma unroll
          for (int i = 0; i < 8; ++i) r[i] = take_term(x[i]);
          if (!LAST) tmem_put_16x16(at + col(0), r);
          if (LAST || (at_once && terms == 3)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = take_term(x[i]);
            if (!LAST) tmem_put_16x16(at + col(1), r);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) r[i] = pack2(x[i]);
          tmem_put_16x16(at + col(LAST || (at_once && terms == 3) ? 2 : 1), r);
        }
      }
      tmem_st_wait();
    };
    constexpr std::integral_constant<bool, false> kAll{};
    constexpr std::integral_constant<bool, true> kThird{};
    // S = lambda^n S + dS (columns past nv hold nothing that is read)
    auto update = [&](int n, int e) {
      if (32 * (warp & 3) < D) {
        const float2 w = tab.step[(n < C ? kLast : kFull) + (e ? kFullLag - kFull : 0)];
        const uint64_t hi = f2(w.x, w.x), low = f2(w.y, w.y);
        float x[32];
        tmem_take16x2(tmem + lane + F::TM_DS + 32 * cg, tmem + lane + F::TM_DS + 32 * cg + 16, x, x + 16);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const uint64_t old = f2(S[i], S[i + 1]);
          f2_out(fma2(hi, old, fma2(low, old, f2(x[i], x[i + 1]))), S[i], S[i + 1]);
        }
      }
    };
    // P: masked, scaled, two bf16 terms in place (each 16 columns: 8 of the first, 8 of the second)
    auto convert_p = [&]() {
      const int tb = 32 * (warp & 3);
#pragma unroll 1
      for (int b = 0; b < F::PW; b += 16) {
        const int s0 = cg * F::PW + b, blk = s0 & ~31;  // a block of 32 x 32: of later positions only, of earlier ones only, or the diagonal
        uint32_t w[16];
        if (blk != tb && (blk > tb) != rev) {
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = 0u;
        } else {
          float x[16];
          tmem_take16(tmem + lane + F::TM_P + s0, x);
          if (blk != tb) {  // lambda^(t - s) = lambda^(t - s0 - 15) lambda^(15 - i)
            const float base = p.a * tab.pw[rev ? s0 - t : t - s0 - 15];
            const uint64_t bb = f2(base, base);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&tab.p16[i]);
              f2_out(mul2(mul2(f2(x[i], x[i + 1]), q.x), bb), x[i], x[i + 1]);
              f2_out(mul2(mul2(f2(x[i + 2], x[i + 3]), q.y), bb), x[i + 2], x[i + 3]);
            }
          } else {
            const int d = t - s0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int k = rev ? i - d : d - i;
              const float v = x[i] * tab.pa[max(k, 0)];
              x[i] = k >= 0 ? v : 0.f;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint64_t v = f2(x[2 * i], x[2 * i + 1]);
            w[i] = take_term(v);
            w[i + 8] = pack2(v);
          }
        }
        tmem_st16(tmem + lane + F::TM_P + s0, w);
      }
      tmem_st_wait();
    };
    // The output rows of a whole chunk, staged over the v tile in its layout for a TMA store
    auto put_tma = [&](int m, int e) {
      const int jj = 32 * cg;
      if (jj < nv) {
        const float f = p.c * tab.pw[(rev ? C - 1 - t : t) + 1 - e];
        const uint64_t ff = f2(f, f);
        const uint32_t st = tile(1, m) + (cg >> 1) * F::ATOM;
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
          float x[16], y[16];
          tmem_take16x2(tmem + lane + F::TM_O1 + jj + j, tmem + lane + F::TM_O2 + jj + j, x, y);
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = pack2(fma2(ff, f2(x[2 * i], x[2 * i + 1]), f2(y[2 * i], y[2 * i + 1])));
          const int ch = 4 * (cg & 1) + j / 8;
          sts128(st + swz_off<128>(t, ch), w[0], w[1], w[2], w[3]);
          sts128(st + swz_off<128>(t, ch + 1), w[4], w[5], w[6], w[7]);
        }
      }
    };
    // The same of any chunk: the warp's 32 rows x 32 columns through its 2 KB of the v tile, to 64-byte pieces of rows
    auto put_out = [&](int m, int e) {
      const int jj = 32 * cg;
      if (jj >= nv) return;
      const int s = rev ? C - 1 - t : t;
      const float f = p.c * tab.pw[s + 1 - e];
      const uint64_t ff = f2(f, f);
      const uint32_t st = tile(1, m) + warp * 2048;
#pragma unroll
      for (int j = 0; j < 32; j += 16) {
        float x[16], y[16];
        tmem_take16x2(tmem + lane + F::TM_O1 + jj + j, tmem + lane + F::TM_O2 + jj + j, x, y);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = pack2(fma2(ff, f2(x[2 * i], x[2 * i + 1]), f2(y[2 * i], y[2 * i + 1])));
        sts128(st + swz_off<64>(ln, j / 8), w[0], w[1], w[2], w[3]);
        sts128(st + swz_off<64>(ln, j / 8 + 1), w[4], w[5], w[6], w[7]);
      }
      __syncwarp();
      const int row = s < left ? decay_row(a, u, p.mode, u.t0 + u.n - left + s) : -1;
      char* o = static_cast<char*>(p.o) + ((size_t)h * p.dv + jj) * 2;
      const size_t os = (size_t)a.H * p.dv * 2;
      const int left = p.dv - jj;
      if (p.dv % 8 == 0) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          const int r = i + ln / 4, gr = __shfl_sync(0xFFFFFFFFu, row, r);
          const uint4 v = lds128(st + swz_off<64>(r, ln & 3));
          if (gr >= 0 && 8 * (ln & 3) < left) *reinterpret_cast<uint4*>(o + gr * os + 16 * (ln & 3)) = v;
        }
      } else {
#pragma unroll 2
        for (int i = 0; i < 32; i += 4) {
          const int r = i + ln / 8, gr = __shfl_sync(0xFFFFFFFFu, row, r);
          const uint2 v = lds64(st + swz_off<64>(r, (ln & 7) >> 1) + 8 * (ln & 1));
          if (gr >= 0 && 4 * (ln & 7) < left) *reinterpret_cast<uint2*>(o + gr * os + 8 * (ln & 7)) = v;
        }
      }
    };

    if constexpr (STATES) {
      // khat of the next chunk is formed while the tensor core sums this one's dS (D = 128: two places for it)
      constexpr bool AHEAD = !F::SMALL;
      const int end = base + same((u.n + C - 1) / C);
#pragma unroll 1
      for (int m = base; m < end + (AHEAD ? 1 : 0); ++m) {
        if (m < end) {
          wait_bar(&sh.full[0][m % F::ST], (m / F::ST) & 1);
          if (__any_sync(0xFFFFFFFFu, timed_out || gone(&sh.abort))) break;
          convert_k(m, terms_of(tab, left - (AHEAD && m > base ? C : 0)), kAll);
        }
        const int j = AHEAD ? m - 1 : m;
        if (!AHEAD) arrive(&sh.bar_k);
        if (j >= base) {
          wait_bar(&sh.bar_ds, j & 1);
          tc_fence_after();
          update(min(C, left), p.lag && u.t0 == 0 && j == base ? 1 : 0);
          left -= C;
        }
        if (AHEAD && m < end) arrive(&sh.bar_k);
      }
      base = end;
      if (t < D) {
        float4* out = block_state(blockIdx.x);
#pragma unroll
        for (int j = 0; j < 32; j += 4) out[(j / 4) * D] = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
      }
    } else {
      auto full = [&](int m) { wait_bar(&sh.full[0][m % F::ST], (m / F::ST) & 1); };
      if (!F::SMALL && left > 0) {
        full(base);
        convert_k(base, terms_of(tab, left), kAll);
      }
      if (!F::SMALL && state) {
        // the state alone: khat of the next chunk is formed while the tensor core sums this one's dS
        arrive(&sh.bar_k);
#pragma unroll 1
        for (int m = base; left > 0; ++m, left -= C) {
          if (__any_sync(0xFFFFFFFFu, timed_out || gone(&sh.abort))) break;
          if (left > C) {
            full(m + 1);
            convert_k(m + 1, terms_of(tab, left - C), kAll);
          }
          wait_bar(&sh.bar_ds, m & 1);
          tc_fence_after();
          update(min(C, left), p.lag && u.t0 == 0 && left == u.n ? 1 : 0);
          arrive(&sh.bar_p);
          arrive(FETCH != kFetchTokens ? &sh.bar_out[m & 1] : &sh.free_[1][m % F::ST]);
          if (left > C) arrive(&sh.bar_k);
        }
        left = 0;
      }
#pragma unroll 1
      for (int m = base; left > 0; ++m, left -= C) {
        const uint32_t ph = m & 1;
        const int n = min(C, left);
        const int e = (p.lag && u.t0 == 0 && left == u.n) ? 1 : 0;
        const int terms = terms_of(tab, left);
        if (F::SMALL) full(m);
        // khat (D = 128: its third term) comes over the last chunk's outputs, once the warps of these lanes have read them.
        // At D = 64 all of them leave together there.  At D = 128 only chunks of three terms have that barrier, and after a
        // wait was given up the warps may learn of it on different sides of the first one: the chunks that are left are
        // passed over, their barriers are not.
        const bool stop = timed_out || gone(&sh.abort);
        if (F::SMALL || terms == 3 ? bar_or(1 + (warp & 3), 32 * CG, stop) : (bool)__any_sync(0xFFFFFFFFu, stop)) {
          if (F::SMALL) break;
          timed_out = true;
          continue;
        }
        if (F::SMALL) convert_k(m, terms, kAll);
        else if (terms == 3) convert_k(m, terms, kThird);
        arrive(&sh.bar_k);
        if (!F::SMALL && !state) {
          wait_bar(&sh.bar_qk, ph);
          tc_fence_after();
          convert_p();
        }
        wait_bar(&sh.bar_ds, ph);
        tc_fence_after();
        if (terms) update(n, e);  // before P v, which comes to stand in dS's place
        if (F::SMALL && !state) {
          wait_bar(&sh.bar_qk, ph);
          tc_fence_after();
          convert_p();
        }
        arrive(&sh.bar_p);
        if (!state) wait_bar(&sh.bar_qs, ph);
        if (left > C && !state) put_state();  // (S_final leaves through the same memory)
        if (!F::SMALL && left > C) {  // while the tensor core is at P v
          full(m + 1);
          convert_k(m + 1, terms_of(tab, left - C), kAll);
        }
        if (!state) {
          wait_bar(&sh.bar_pv, ph);
          tc_fence_after();
          if (FETCH != kFetchTokens && n == C) put_tma(m, e);
          else put_out(m, e);
        }
        arrive(FETCH != kFetchTokens ? &sh.bar_out[m & 1] : &sh.free_[1][m % F::ST]);  // (the tile is stored from, or fetched over)
      }
      base += same((u.n + C - 1) / C);
      if (tab.publish) {  // to the blocks that go on
        if (t < D) {
          float4* out = block_state(sh.me);
#pragma unroll
          for (int j = 0; j < 32; j += 4) out[(j / 4) * D] = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
        }
        __threadfence();
        named_bar(9, NT);
        if (tid == 0) asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(a.flag + sh.me), "r"(1u) : "memory");
      }
      if (tab.keep && u.last && 32 * (warp & 3) < D) {
        // dS0 = lambda G_0; an empty sequence passes its state on as it is
        const float w = p.lag && u.len > 0 ? tab.pw[1] : 1.f;
        float* out = p.Sf + ((size_t)u.slot * a.H + h) * p.dk * p.dv;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 16 * half + 4 * i;
            sts128(stage + swz_off<64>(ln, i), __float_as_uint(w * S[j]), __float_as_uint(w * S[j + 1]), __float_as_uint(w * S[j + 2]), __float_as_uint(w * S[j + 3]));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = lds128(stage + swz_off<64>(8 * i + ln / 4, ln & 3));
            if (state_in(8 * i + ln / 4, half))
              *state_at(out, 8 * i + ln / 4, half) = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
          }
          __syncwarp();
        }
      }
    }
    if (!piece_done()) break;
    }
  }
  if (timed_out) set_status(a.status, DIG_ERR_DEVICE_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W0) tmem_dealloc(tmem, F::TM_COLS);
  if (a.deal.handoff) {  // the last block to end leaves counters and flags as they were
    if (tid == 0) sh.abort = atomicAdd(a.counter + 1, 1u) == gridDim.x - 1;
    __syncthreads();
    if (sh.abort) {
      for (int i = tid; i < a.deal.grid; i += NT + 128) a.flag[i] = 0u;
      if (tid < 2) a.counter[tid] = 0u;
    }
  }
}

// The states that the first pass left, joined in place: block i's then is its unit's state up to the end of its run.
template <int D>
__global__ void __launch_bounds__(256) decay_join_kernel(const __grid_constant__ DecayArgs a) {
  __shared__ float2 step[2];
  griddep_wait();
  griddep_launch_dependents();
  const long long per = (long long)a.B * a.deal.chunks, start = (long long)blockIdx.x * a.deal.chunks;
  const DealRuns runs(per * a.H * a.deal.nprob, a.deal.grid);
  const int j0 = runs.block_of(start), j1 = runs.block_of(start + a.deal.chunks - 1);  // the last one's is not needed
  const long long zh = deal_div(blockIdx.x, a.B);
  if (threadIdx.x < 2) step[threadIdx.x] = decay_pow(a.g[zh % a.H], (runs.q + threadIdx.x) * C);
  __syncthreads();
  float4* s = reinterpret_cast<float4*>(a.segst) + blockIdx.y * 256 + threadIdx.x;
  constexpr int STATE = D * D / 4;
  if (j1 - j0 < 2) return;
  float4 S = s[(size_t)j0 * STATE];
  for (int i0 = j0 + 1; i0 < j1; i0 += 8) {
    float4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = s[(size_t)min(i0 + i, j1 - 1) * STATE];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i0 + i < j1) {
        const float2 w = step[i0 + i < runs.rem];
        S.x = fmaf(w.x, S.x, fmaf(w.y, S.x, x[i].x));
        S.y = fmaf(w.x, S.y, fmaf(w.y, S.y, x[i].y));
        S.z = fmaf(w.x, S.z, fmaf(w.y, S.z, x[i].z));
        S.w = fmaf(w.x, S.w, fmaf(w.y, S.w, x[i].w));
        s[(size_t)(i0 + i) * STATE] = S;
      }
  }
}

template <int D, bool STATES, int FETCH>
cudaError_t run(const DecayArgs& a, cudaStream_t s) {
  using F = TcCfg<D, STATES>;
  constexpr int smem = F::OFF_T + sizeof(TcTables<F::ST>);
  static std::atomic<uint64_t> set{0};  // devices whose kernel has its shared memory allowed
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && !(dev < 64 && (set.load(std::memory_order_relaxed) >> dev & 1))) {
    e = cudaFuncSetAttribute(decay_tc_kernel<D, STATES, FETCH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) set.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(decay_tc_kernel<D, STATES, FETCH>, dim3(a.deal.grid), dim3(F::NT + 128), smem, s, a);
}

template <int D, int FETCH>
cudaError_t passes(const DecayArgs& a, cudaStream_t s) {
  cudaError_t e;
  if (a.deal.joined && (e = run<D, true, FETCH>(a, s)) != cudaSuccess) return e;
  if (a.deal.joined &&
      (e = launch_pdl(decay_join_kernel<D>, dim3(a.B * a.H * a.deal.nprob, D * D / 1024), dim3(256), 0, s, a)) != cudaSuccess)
    return e;
  return run<D, false, FETCH>(a, s);
}

}  // namespace

cudaError_t launch_decay_tc(const DecayArgs& a, int D, cudaStream_t s) {
  auto go = [&](auto d) {
    constexpr int DD = decltype(d)::value;
    return a.fetch == kFetchRows   ? passes<DD, kFetchRows>(a, s)
           : a.fetch == kFetchCols ? passes<DD, kFetchCols>(a, s)
                                   : passes<DD, kFetchTokens>(a, s);
  };
  return D == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

}  // namespace dig
