// kda_linear_tile.cu -- linear attention with a decay for each head, whole
// prompts on the tensor cores (bf16, dk and dv 64 or 128).
//
// In chunks of 128 tokens, with G_i the sum of the log-decays of a chunk's
// tokens 0 .. i, E its last and S the state before it:
//
//   O  = diag(e^G) (Q S) + P V,      P_ij = e^(G_i - G_j) (q_i . k_j), j <= i
//   S' = e^E S + K^T V',             V'_j = e^(E - G_j) v_j
//
// A CTA takes items (a sequence or a segment of one, a head, 64 value columns)
// and walks their chunks, its state S in registers (fp32); Q K^T, P V, Q S and
// K^T V' are tcgen05 products into tensor memory.  One warp feeds Q, K and V by
// TMA (two or three chunks ahead), one issues products, two take the decays' sums, and
// sixteen do the same work side by side, each a quarter of the rows and a fourth
// of the columns: V', S and its operand, P, O.  The products of a chunk run in
// the order Q S, K^T V', P V, the next chunk's scores; while each runs, the
// sixteen work on what the one before it left.  (With groups of warps for P, S,
// V' and O the same work took 1.5 to 2 times as long: four kinds of loops on
// each scheduler do not fit its instruction caches.)
//
// Rounding: P and the state as an operand enter as bf16, as the tensor cores multiply
// V's 16 bits by nothing wider, and tensor memory and shared memory are full without
// second parts of them: each is one rounding of 2^-9 beside the output's own
// (outputs err by 2.3e-3 of their norm, the roundings of the outputs alone are
// 1.7e-3).  Rows of Q keep their bits, e^G being applied to the product.  The state
// itself is summed from V' in three bf16 parts, which hold all of its 24 bits: what is
// carried and returned is fp32 (1.2e-7 of its norm from 64 bits, as plain 32-bit
// operations; two parts left 2.4e-6, and took 0.9 of the time of a full chip's prompts
// and 0.85 of a first pass).  Sums of log-decays are exact, in fixed point, as their
// differences are what counts.  Where a tile lies below the diagonal
// of 32-token blocks, e^(G_i - G_j) is e^(G_i - G_b) e^(G_b - G_j) with b the
// last token of j's block: both factors are at most 1, so neither overflows
// and the product only vanishes where the weight does.
//
// Few items (long rows of few heads) would leave SMs idle: sequences are then
// cut into segments.  A first pass sums each segment's own state (no Q, no
// output), a scan composes the states that segments start from, and the full
// pass runs every segment at once.
//
// Measured: two rows of 32 768 tokens, 32 heads of 128 channels, 502 us, 4.3 TB/s
// (0.64 of a copy's); 17 ragged prompts, 16 heads, 156 us; one row of 131 072
// tokens, 16 heads, 726 us (250 of them the first pass).  A chunk takes some 3900
// cycles, the products 2000 of them.
#include <cudaTypedefs.h>

#include "kda_cache_attn.cuh"
#include "kda_linear.cuh"
#include "kda_tc_util.cuh"

namespace {

using namespace kda_linear;
using kda_cache::kernel_may_follow;
using kda_cache::launch_following;
using kda_cache::wait_for_kernel_before;

constexpr int C = 128;          // tokens of a chunk
constexpr int NV = 64;          // value columns of a CTA
constexpr int kThreads = 640;
// tensor memory: scores, P, Q S by stage, P V, K^T V' of the first part of V' and of the others
constexpr uint32_t TM_S = 0, TM_P = 128, TM_O1 = 192, TM_O2 = 320, TM_DS = 384, kTmemCols = 512;
// in the first pass: K^T V' of V's three parts, of even and of odd chunks
constexpr uint32_t TM_D0 = 0, TM_D1 = 192;
constexpr int kWorkers = kThreads / 32 - 4;

struct TileArgs {
  LinearArgs a;
  int seg;         // tokens of a segment, a multiple of C (longer than any sequence: none)
  int segs;        // dense: segments of a sequence
  int cols;        // (sequence, segment) columns; packed: the most there can be
  int halves;      // dv / NV
  float* states;   // [cols, H, dk, dv]: what segments end with (first pass), then start from
  float2* gammas;  // [cols, H] a segment's decay factor, in two parts (-1, 0: it forgets)
};

// What a chunk's decays come to (G: sums of log2-decays).
struct alignas(16) Gate {
  float back[C];   // G_b - G_j, b the last token of j's 32
  float col[C];    // 2^(G_b - G_j)
  float tail[4];   // 2^(E - G_b) of each 32
  int2 end[4];     // G_b of each 32, in units of 2^-16 and 2^-40
};
struct alignas(16) Total {
  float gamma[2];  // 2^E in two parts
  int first;       // the first token that forgets, C if there is none
  int unused;
};
constexpr int kTotals = 4;  // (read until the chunk's rows go out; the next but three comes later)

// A wait tells a phase only from its neighbours, so every waiter takes every phase of its
// barrier in turn, and none can end before all have passed the one before it; why, beside each.
struct Bars {
  uint64_t qk_full[3], v_full[2];    // copies have landed (the next into the same place waits for
                                     // ds_done, o_done or, V in the first pass, ready: so for V'
                                     // and P, made by all behind their waits for it)
  uint64_t ds_done[3];               // K^T V' and Q S are there: V', K, Q and S's operand are free
                                     // (the next of a place needs its K, so the copies' warp, and
                                     // `ready`, which the sixteen give behind theirs)
  uint64_t o_done[2];                // P V is there: V and P are free (likewise, by V and p_full)
  uint64_t s_done;                   // the scores are there (the next ones come behind p_full)
  uint64_t ready[2];                 // V' and S's operand are made, K^T V' and Q S's places read
                                     // (given again behind ds_done of a chunk that it let begin)
  uint64_t p_full;                   // P is made, the scores and P V's place read (given again
                                     // behind s_done, which follows the wait for it)
  uint64_t gate_full[2], gate_empty[2];  // (each needs the other's last one)
  uint64_t drain;
};

// The full pass: Q, K and V in two stages, V' and S's operand.  The first pass: K in three
// stages, V in two (free as soon as V' is made), V' in two places.  At 128 channels each takes
// all that a CTA can have but 250 bytes.
template <int DK, bool OUT>
struct Smem {
  static constexpr int kStages = OUT ? 2 : 3;
  static constexpr int kTile = C * DK * 2;                 // Q or K of a chunk
  static constexpr int kBox = C * 128;                     // 64 channels of it
  static constexpr int kQ = 0, kK = OUT ? 2 * kTile : 0, kV = kK + kStages * kTile;
  static constexpr int kVP = kV + 2 * kBox;                // V' in three parts
  static constexpr int kVP1 = OUT ? kVP : kVP + 3 * kBox;  // the same of odd chunks
  static constexpr int kS = kVP1 + 3 * kBox;               // S as an operand
  static constexpr int kGate = kS + (OUT ? DK * NV * 2 : 0);
  static constexpr int kTotal = kGate + 2 * (int)sizeof(Gate);
  static constexpr int kBars = kTotal + kTotals * (int)sizeof(Total);
  static constexpr int kOrder = kBars + (int)sizeof(Bars) + 16;
  // most sequences of a packed batch that are put in order
  static constexpr int kOrdered = DK == 64 ? 1024 : 320;
  static constexpr int kBytes = kOrder + 2 * kOrdered;
  static_assert(kBytes <= 232448, "more than a CTA can have");
};

// Items go to the CTAs there and back: round by round, every other one from the
// last CTA to the first, so that with the longest first all get about as much.
__device__ __forceinline__ int following(int id) {
  const int G = gridDim.x, round = id / G;
  return (2 * round + 2) * G - 1 - id;
}

struct Item {
  int64_t row;  // first token row
  int len;      // tokens
  int n, h, hk, half, col;
  int tail;     // column of its sequence's last segment
  bool first, last;  // segment of its sequence
};

// Item `id` of the grid's; false: there is none of that number (packed columns
// are as many as there can be), or nothing to do in this pass.
template <bool OUT>
__device__ __noinline__ bool locate(const TileArgs& p, const uint16_t* order, int id, Item& it) {
  const int x = id / p.halves;
  it.half = id - x * p.halves;
  it.col = x / p.a.H;
  it.h = x - it.col * p.a.H;
  it.hk = it.h / (p.a.H / p.a.HK);
  int seg;
  if (!p.a.cu) {
    it.n = it.col / p.segs;
    seg = it.col - it.n * p.segs;
  } else {
    // sequence n has the columns cu[n] / seg + n and up: as many as it has
    // segments, and at most one more
    int lo = 0, hi = p.a.N - 1;
    if (p.seg > p.a.T) {
      lo = order ? order[it.col] : it.col;
    } else {
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.a.cu[mid] / p.seg + mid <= it.col) lo = mid;
        else hi = mid - 1;
      }
    }
    it.n = lo;
    seg = p.seg > p.a.T ? 0 : it.col - (p.a.cu[lo] / p.seg + lo);
  }
  int64_t row;
  int len;
  if (!span(p.a, it.n, row, len)) return false;
  const int segs = len == 0 ? 1 : (len + p.seg - 1) / p.seg;
  if (seg < 0 || seg >= segs) return false;
  it.first = seg == 0;
  it.last = seg == segs - 1;
  it.tail = it.col + segs - 1 - seg;
  if (!OUT && it.last) return false;
  it.row = row + (int64_t)seg * p.seg;
  it.len = it.last ? len - seg * p.seg : p.seg;
  return true;
}

// The chunks of a CTA's items, one after the other.
template <bool OUT>
struct Walk {
  const TileArgs& p;
  const uint16_t* order;
  int id, ids;
  Item it;
  int t;       // first token of the chunk in its item
  bool valid;
  __device__ __forceinline__ Walk(const TileArgs& args, const uint16_t* ord, bool begin = true)
      : p(args), order(ord), id(blockIdx.x), ids(args.cols * args.a.H * args.halves), t(0),
        valid(false) {
    if (begin) settle();
  }
  __device__ __forceinline__ bool find() {
    Item x;  // (the call's copy is in memory, this one's in registers)
    const bool there = locate<OUT>(p, order, id, x);
    it = x;
    return there;
  }
  __device__ __forceinline__ void settle() {
    for (; id < ids; id = following(id))
      if (find() && it.len > 0) break;
    valid = id < ids;
    t = 0;
  }
  __device__ __forceinline__ void next() {
    t += C;
    if (t < it.len) return;
    id = following(id);
    settle();
  }
  __device__ __forceinline__ int rows() const { return it.len - t < C ? it.len - t : C; }
};

// A fixed-point number of units of 2^-16 and 2^-40.
__device__ __forceinline__ float fixed(int hi, int lo) {
  return fmaf((float)lo, 1.0f / 1099511627776.0f, (float)hi * (1.0f / 65536.0f));
}
__device__ __forceinline__ void tmem_st8(uint32_t ta, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(ta),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
               "r"(r[7])
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Products are issued by a whole warp that runs in step, of which one thread
// (`one`) carries them out: so their operands are known to be uniform, and a
// product issues at the tensor cores' own rate.  Four k-steps; the descriptors'
// low words (16-byte units) go up by AS and BS a step.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(r));
  return r;
}
template <int AS, int BS>
__device__ __forceinline__ void mma4_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t a_hi,
                                        uint32_t b_hi, uint32_t idesc, uint32_t accumulate,
                                        uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b64 a, b;\n .reg .b32 x, y;\n"
      " setp.ne.b32 q, %7, 0;\n setp.ne.b32 p, %6, 0;\n setp.eq.b32 t, 0, 0;\n"
      " mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n"
      " add.u32 x, %1, %8;\n add.u32 y, %2, %9;\n mov.b64 a, {x, %3};\n mov.b64 b, {y, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n"
      " add.u32 x, %1, 2 * %8;\n add.u32 y, %2, 2 * %9;\n mov.b64 a, {x, %3};\n"
      " mov.b64 b, {y, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n"
      " add.u32 x, %1, 3 * %8;\n add.u32 y, %2, 3 * %9;\n mov.b64 a, {x, %3};\n"
      " mov.b64 b, {y, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(one), "n"(AS),
      "n"(BS)
      : "memory");
}
// A in tensor memory, 8 columns a step
template <int BS>
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi,
                                        uint32_t idesc, uint32_t accumulate, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b64 b;\n .reg .b32 x, y;\n"
      " setp.ne.b32 q, %6, 0;\n setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, 0, 0;\n"
      " mov.b64 b, {%2, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n"
      " add.u32 x, %1, 8;\n add.u32 y, %2, %7;\n mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n"
      " add.u32 x, %1, 16;\n add.u32 y, %2, 2 * %7;\n mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n"
      " add.u32 x, %1, 24;\n add.u32 y, %2, 3 * %7;\n mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(one), "n"(BS)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(
          sm100::smem_u32(bar)),
      "r"(one)
      : "memory");
}

// Bounded wait (2 s), which also gives up when another role of the CTA has.  The
// hint lets the hardware suspend the warp for up to 1 ms: one that polls takes
// issue slots and shared memory's from those that work.
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000000)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  const uint64_t t0 = sm100::globaltimer_ns();
  while (!poll(bar, parity))
    if (*abort || sm100::globaltimer_ns() - t0 > 2000000000ull) {
      *abort = 1;
      return false;
    }
  return true;
}

// Two fp32 at a time.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(f32x2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(f32x2 x) {
  float a, b;
  unpair(x, a, b);
  return sm100::pack_bf16x2(a, b);
}

template <int DK, bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
    kda_linear_tile_kernel(const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v,
                           const __grid_constant__ TileArgs p) {
  using M = Smem<DK, OUT>;
  constexpr uint32_t NS = M::kStages;
  // (the copies' swizzle goes by addresses of 1024 bytes)
  extern __shared__ __align__(1024) unsigned char smem[];
  Gate* gates = reinterpret_cast<Gate*>(smem + M::kGate);
  Total* totals = reinterpret_cast<Total*>(smem + M::kTotal);
  Bars& bars = *reinterpret_cast<Bars*>(smem + M::kBars);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + M::kBars + sizeof(Bars));
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!OUT) kernel_may_follow();

  if (warp == 1) {
    sm100::tmem_alloc(s_tmem, kTmemCols);
    sm100::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      sm100::mbar_init(&bars.qk_full[i], 1);
      sm100::mbar_init(&bars.ds_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&bars.v_full[i], 1);
      sm100::mbar_init(&bars.gate_full[i], 1);
      sm100::mbar_init(&bars.gate_empty[i], kWorkers);
      sm100::mbar_init(&bars.o_done[i], 1);
      sm100::mbar_init(&bars.ready[i], kWorkers);
    }
    sm100::mbar_init(&bars.s_done, 1);
    sm100::mbar_init(&bars.p_full, kWorkers);
    sm100::mbar_init(&bars.drain, 1);
    sm100::fence_mbar_init();
    *s_abort = 0;
  }
  // whole sequences of a packed batch: the longest first, equal ones in order.  (Lengths of
  // malformed offsets are some numbers too: every sequence gets a place of its own.)
  uint16_t* order = nullptr;
  if (p.a.cu && p.seg > p.a.T && p.a.N <= M::kOrdered) {
    order = reinterpret_cast<uint16_t*>(smem + M::kOrder);
    int* lens = reinterpret_cast<int*>(smem + M::kVP);  // (where V' comes later)
    const int N4 = (p.a.N + 3) / 4;
    for (int n = tid; n < 4 * N4; n += kThreads)
      lens[n] = n < p.a.N ? (int)((uint32_t)p.a.cu[n + 1] - (uint32_t)p.a.cu[n]) : INT32_MIN;
    __syncthreads();
    for (int n = tid; n < p.a.N; n += kThreads) {
      const int len = lens[n];
      int rank = 0;
      for (int m = 0; m < N4; ++m) {
        const int4 x = reinterpret_cast<const int4*>(lens)[m];
        rank += (x.x > len || (x.x == len && 4 * m < n)) +
                (x.y > len || (x.y == len && 4 * m + 1 < n)) +
                (x.z > len || (x.z == len && 4 * m + 2 < n)) +
                (x.w > len || (x.w == len && 4 * m + 3 < n));
      }
      order[rank] = (uint16_t)n;
    }
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  // (the whole of tensor memory is this CTA's: its columns count from 0)
  const uint32_t tmem = 0;

  // The barrier's phase n.  The warp's threads leave together and with one answer: what comes
  // next (loads and stores of tensor memory, shuffles, products) is for whole warps, and a wait
  // that gives up ends the role for all of them.  (One vote where the phase is over, on which all
  // then branch: with the vote behind both ways the two rows took 464 us, so 456, with none 453.)
  auto wait = [&](uint64_t* bar, uint32_t n) -> bool {
    const uint32_t at = sm100::smem_u32(bar);
    if (__all_sync(~0u, poll(at, n & 1))) return true;
    return __all_sync(~0u, bounded_wait(at, n & 1, s_abort));
  };
  // a warp's arrival, after all of its threads' work before it
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(bar);
  };

  if (warp == 0) {
    // ------------------------------------------------------ Q, K and V come
    uint32_t g = 0;
    auto load_v = [&](const Item& it, int row, uint32_t g) {
      sm100::mbar_arrive_expect_tx(&bars.v_full[g & 1], M::kBox);
      sm100::tma_load_3d(smem + M::kV + (g & 1) * M::kBox, &map_v, &bars.v_full[g & 1], NV * it.half,
                         it.h, row);
    };
    for (Walk<OUT> w(p, order); w.valid; w.next(), ++g) {
      const uint32_t s = g % NS, use = g / NS;
      const int row = (int)(w.it.row + w.t), hk = w.it.hk;
      // (in the order in which their places become free)
      if (!OUT && g > 1 && !wait(&bars.ready[g & 1], (g >> 1) - 1)) break;
      if (!OUT && lane == 0) load_v(w.it, row, g);
      if (use > 0 && !wait(&bars.ds_done[s], use - 1)) {
        if (!OUT) ++g;
        break;
      }
      if (lane == 0) {
        sm100::mbar_arrive_expect_tx(&bars.qk_full[s], (OUT ? 2 : 1) * M::kTile);
#pragma unroll
        for (int b = 0; b < DK / 64; ++b) {
          const int at = s * M::kTile + b * M::kBox;
          sm100::tma_load_3d(smem + M::kK + at, &map_k, &bars.qk_full[s], 64 * b, hk, row);
          if (OUT) sm100::tma_load_3d(smem + M::kQ + at, &map_q, &bars.qk_full[s], 64 * b, hk, row);
        }
      }
      __syncwarp();
      // (a give-up leaves one of the chunk's copies out: nobody gets beyond its barrier)
      if (OUT && use > 0 && !wait(&bars.o_done[s], use - 1)) {
        ++g;
        break;
      }
      if (OUT && lane == 0) load_v(w.it, row, g);
      __syncwarp();
    }
    // copies in flight end before the CTA does
    for (uint32_t i = g < NS ? 0 : g - NS; i < g; ++i)
      sm100::mbar_wait(&bars.qk_full[i % NS], (i / NS) & 1, 200000000ull);
    for (uint32_t i = g < 2 ? 0 : g - 2; i < g; ++i)
      sm100::mbar_wait(&bars.v_full[i & 1], (i >> 1) & 1, 200000000ull);
  } else if (warp == 1) {
    // ----------------------------------------------------------- products
    const uint32_t one = elect_one();
    constexpr uint32_t id_s = sm100::idesc_bf16(C, C, 0, 0), id_q = sm100::idesc_bf16(C, NV, 0, 1);
    constexpr uint32_t id_d = sm100::idesc_bf16(DK, (OUT ? 2 : 3) * NV, 1, 1);
    constexpr uint32_t id_d2 = sm100::idesc_bf16(DK, NV, 1, 1);
    // (addresses in a descriptor count 16 bytes; a box of 64 channels is one span along M or N)
    constexpr uint32_t kTile16 = M::kTile / 16, kBox16 = M::kBox / 16;
    const uint32_t at = (uint32_t)sm100::smem_desc(sm100::smem_u32(smem), M::kBox, 1024);
    const uint32_t hi = (uint32_t)(sm100::smem_desc_sw128(0, M::kBox, 1024) >> 32);
    const uint32_t dq = at + M::kQ / 16, dk = at + M::kK / 16, dv = at + M::kV / 16;
    // (the first pass has V' and its product twice, by odd and even chunks)
    const uint32_t dvp = at + M::kVP / 16, dvp1 = at + M::kVP1 / 16;
    const uint64_t st = sm100::smem_desc(sm100::smem_u32(smem) + M::kS, 1024, 128);
    const uint32_t dst = (uint32_t)st, st_hi = (uint32_t)(st >> 32);
    // every thread takes the same way (and the compiler knows)
    auto all = [&](bool x) -> bool { return __all_sync(~0u, x); };
    auto scores = [&](uint32_t s) {
#pragma unroll
      for (int b = 0; b < DK / 64; ++b)
        mma4_ss<2, 2>(TM_S, dq + s * kTile16 + b * kBox16, dk + s * kTile16 + b * kBox16, hi, hi,
                      id_s, b, one);
      commit(&bars.s_done, one);
    };
    uint32_t g = 0;
    Walk<OUT> w(p, order);
    bool more = all(w.valid);
    if (OUT && more) {
      more = wait(&bars.qk_full[0], 0);
      sm100::tc_fence_after();
      if (more) scores(0);
    }
    // chunk g; false: the last one, or a wait gave up
    auto chunk = [&]() -> bool {
      const uint32_t s = g % NS, odd = g & 1;
      if (!OUT && !wait(&bars.qk_full[s], g / NS)) return false;
      if (!wait(&bars.ready[odd], g >> 1)) return false;
      sm100::tc_fence_after();
      if (OUT) {
#pragma unroll
        for (uint32_t b = 0; b < DK / 64; ++b)
          mma4_ss<2, 128>(TM_O1 + NV * s, dq + s * kTile16 + b * kBox16, dst + 512 * b, hi, st_hi,
                          id_q, b, one);
      }
      // (in the full pass V's third part is added to what the second gives: tensor memory is full)
      const uint32_t to = OUT ? TM_DS : odd ? TM_D1 : TM_D0, from = odd ? dvp1 : dvp;
#pragma unroll
      for (uint32_t k = 0; k < 2; ++k)
        mma4_ss<128, 128>(to, dk + s * kTile16 + 512 * k, from + 512 * k, hi, hi, id_d, k, one);
#pragma unroll
      for (uint32_t k = 0; OUT && k < 2; ++k)
        mma4_ss<128, 128>(to + NV, dk + s * kTile16 + 512 * k, from + 2 * kBox16 + 512 * k, hi, hi,
                          id_d2, 1, one);
      commit(&bars.ds_done[s], one);
      w.next();
      const bool next = all(w.valid);
      if (OUT) {
        if (!wait(&bars.p_full, g)) return false;
        sm100::tc_fence_after();
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k)
          mma4_ts<128>(TM_O2, TM_P + 32 * k, dv + s * kBox16 + 512 * k, hi, id_q, k, one);
        commit(&bars.o_done[s], one);
        if (next) {
          if (!wait(&bars.qk_full[s ^ 1], (g + 1) >> 1)) return false;
          sm100::tc_fence_after();
          scores(s ^ 1);
        }
      }
      ++g;
      return next;
    };
    while (more) more = chunk();
    commit(&bars.drain, one);
    sm100::mbar_wait(&bars.drain, 0, 200000000ull);
  } else if (warp < 4) {
    // --------------------- sums of the log-decays: two warps, chunks in turn
    const uint32_t turn = warp - 2;
    // malformed offsets of any sequence: with segments, a search may pass one by
    if (OUT && turn && p.a.cu && p.seg <= p.a.T && blockIdx.x == 0)
      for (int n = lane; n < p.a.N; n += 32) {
        int64_t row;
        int len;
        span(p.a, n, row, len);
      }
    // the log-decays of a chunk, four tokens a lane
    auto fetch = [&](const Walk<OUT>& w, float (&y)[4]) {
      const float* a = p.a.decay + (w.it.row + w.t) * p.a.decay_stride + w.it.h;
      const int L = w.rows();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 4 * lane + e;
        y[e] = t < L ? a[t * p.a.decay_stride] : 0.0f;
      }
    };
    Walk<OUT> w(p, order);
    if (turn && w.valid) w.next();
    float y[4];
    if (w.valid) fetch(w, y);
    for (uint32_t g = turn; w.valid; g += 2) {
      const int L = w.rows();
      // fixed point, exact in its sums: 2^-16 and 2^-40 a unit
      int hi[4], lo[4], sum_hi = 0, sum_lo = 0;
      uint32_t nan = 0, cut = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // 2^-160 vanishes in 32 bits: what decays more than that decays so much
        const float c = clamp_decay(y[e]) * 1.4426950408889634f, x = c < -160.0f ? -160.0f : c;
        nan |= (x != x) << e;
        cut |= forgets(y[e]) << e;
        const int i = __float2int_rn(x * 65536.0f);
        hi[e] = sum_hi += i;
        lo[e] = sum_lo += __float2int_rn(fmaf((float)i, -1.0f / 65536.0f, x) * 1099511627776.0f);
      }
      // (the next ones on their way meanwhile)
      w.next();
      if (w.valid) w.next();
      if (w.valid) fetch(w, y);
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int a = __shfl_up_sync(~0u, sum_hi, d), b = __shfl_up_sync(~0u, sum_lo, d);
        if (lane >= d) sum_hi += a, sum_lo += b;
      }
      const int end_hi = __shfl_sync(~0u, sum_hi, 31), end_lo = __shfl_sync(~0u, sum_lo, 31);
      const int blk_hi = __shfl_sync(~0u, sum_hi, lane | 7), blk_lo = __shfl_sync(~0u, sum_lo, lane | 7);
      const int pre_hi = sum_hi - hi[3], pre_lo = sum_lo - lo[3];
      // a NaN makes what follows it NaN
      const uint32_t bad = __ballot_sync(~0u, nan != 0), cuts = __ballot_sync(~0u, cut != 0);
      const int at = __ffs(cuts) - 1, first = cuts ? 4 * at + __ffs(__shfl_sync(~0u, cut, at)) - 1 : C;
      float back[4], col[4];
      const float none = __int_as_float(0x7fffffff);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int h = pre_hi + hi[e], l = pre_lo + lo[e];
        back[e] = fixed(blk_hi - h, blk_lo - l);
        col[e] = ex2(back[e]);
        // (rare) no sum for tokens from the first NaN on
        if (bad && ((bad & ((1u << lane) - 1)) || (nan & ((2u << e) - 1)))) back[e] = none;
      }
      // (and no weight to the chunk's end)
      const float tail = bad ? none : ex2(fixed(end_hi - blk_hi, end_lo - blk_lo));
      // close to 1, as 1 + (2^E - 1) and what that lost (see the kernel for single tokens)
      const float x = fixed(end_hi, end_lo) * 0.6931471805599453f;
      const float m = expm1f(x), f = 1.0f + m;
      const float2 gamma = bad         ? make_float2(none, none)
                           : x > -0.5f ? make_float2(f, m - (f - 1.0f))
                                       : make_float2(expf(x), 0.0f);
      if (g > 1 && !wait(&bars.gate_empty[turn], (g >> 1) - 1)) break;
      Gate& gate = gates[turn];
      reinterpret_cast<float4*>(gate.back)[lane] = make_float4(back[0], back[1], back[2], back[3]);
      reinterpret_cast<float4*>(gate.col)[lane] = make_float4(col[0], col[1], col[2], col[3]);
      if ((lane & 7) == 7) {
        gate.end[lane >> 3] = make_int2(blk_hi, blk_lo);
        gate.tail[lane >> 3] = tail;
      }
      if (lane == 0)
        *reinterpret_cast<float4*>(&totals[g % kTotals]) =
            make_float4(gamma.x, gamma.y, __int_as_float(first), 0.0f);
      // Rows past a sequence's end belong to others: zeros, whatever they hold.  (This warp's
      // chunks are those of one stage, and it sees each of its copies land: no phase is missed.
      // Segments of the first pass are whole chunks.)
      if (OUT) {
        const uint32_t s = g & 1;
        if (!wait(&bars.qk_full[s], g >> 1) || !wait(&bars.v_full[s], g >> 1)) break;
        if (L < C) {
          const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 1
          for (int e = L * 8 + lane; e < C * 8; e += 32) {
#pragma unroll
            for (int b = 0; b < DK / 64; ++b)
              reinterpret_cast<uint4*>(smem + M::kK + s * M::kTile + b * M::kBox)[e] = zero;
            reinterpret_cast<uint4*>(smem + M::kV + s * M::kBox)[e] = zero;
          }
          sm100::fence_async_smem();
        }
      }
      arrive(&bars.gate_full[turn]);
    }
  } else {
    // ------ sixteen warps that all do a quarter's fourth of V', S, P and O in turn
    const int q = warp & 3, part = (warp >> 2) - 1, row = 32 * q + lane;
    const int c0 = 16 * part;  // value columns c0 .. c0 + 15 of S and O
    // (a product of 64 rows has them in the first half of each warp's lanes)
    const int i = DK == 128 ? row : 16 * q + lane;
    const bool mine = DK == 128 || lane < 16;
    const uint32_t tm = sm100::taddr(tmem, 32 * q, 0);
    const bool whole = (reinterpret_cast<uint64_t>(p.a.out) & 31) == 0;
    f32x2 S[8];
    float* to = nullptr;  // where the item's state goes
    double all = 1.0;     // a segment's decay
    bool gone = false;    // it forgets
    Item it{};
    int id = blockIdx.x, t = 0;
    auto leave = [&]() {
      if (to && mine)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          float4 x;
          unpair(S[j / 2], x.x, x.y);
          unpair(S[j / 2 + 1], x.z, x.w);
          *reinterpret_cast<float4*>(to + j) = x;
        }
      if (!OUT && it.half == 0 && tid == 128) {
        const float hi = (float)all;
        p.gammas[(int64_t)it.col * p.a.H + it.h] =
            gone ? make_float2(-1.0f, 0.0f) : make_float2(hi, (float)(all - (double)hi));
      }
    };
    // the next item with tokens, from id on: its entry state (an empty sequence's state passes)
    auto enter = [&]() -> bool {
      const int ids = p.cols * p.a.H * p.halves;
      for (; id < ids; id = following(id)) {
        Item x;
        if (!locate<OUT>(p, order, id, x)) continue;
        it = x;
        const int64_t size = (int64_t)DK * p.a.dv, unit = (int64_t)it.n * p.a.H + it.h;
        const int64_t in = (int64_t)i * p.a.dv + NV * it.half + c0;
        const int64_t col = (int64_t)it.col * p.a.H + it.h;
        // (final_state may be init_state: where other segments follow, the first one of the full
        // pass starts from the copy that the scan has left in the last one's place)
        const float* from =
            !it.first              ? (OUT ? p.states + (col - p.a.H) * size : nullptr)
            : OUT && it.tail != it.col ? p.states + ((int64_t)it.tail * p.a.H + it.h) * size
            : p.a.init             ? p.a.init + unit * size
                                   : nullptr;
        to = !OUT      ? p.states + col * size
             : it.last ? (p.a.final_state ? p.a.final_state + unit * size : nullptr)
                       : nullptr;
        if (to) to += in;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 x = from && mine ? *reinterpret_cast<const float4*>(from + in + j)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
          S[j / 2] = pair(x.x, x.y);
          S[j / 2 + 1] = pair(x.z, x.w);
        }
        t = 0;
        all = 1.0;
        gone = false;
        if (it.len > 0) return true;
        leave();
      }
      return false;
    };
    // V' of chunk g, 16 bytes a thread at a time (rows of V past the end are zeros by then).
    auto weigh = [&](uint32_t g) -> bool {
      if (!wait(&bars.gate_full[g & 1], g >> 1)) return false;  // (in the full pass V is there)
      const Gate& gate = gates[g & 1];
      if (!OUT && !wait(&bars.v_full[g & 1], g >> 1)) return false;
      const uint4* v = reinterpret_cast<const uint4*>(smem + M::kV + (g & 1) * M::kBox);
      uint4* to = reinterpret_cast<uint4*>(smem + (g & 1 ? M::kVP1 : M::kVP));
      const f32x2 minus = pair(-1.0f, -1.0f);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = 512 * k + tid - 128;
        const uint4 x = v[e];
        const float f = gate.col[e >> 3] * gate.tail[e >> 8];
        const f32x2 ff = pair(f, f);
        const uint32_t r[4] = {x.x, x.y, x.z, x.w};
        uint32_t a[4], b[4], d[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          auto two = [](uint32_t w) {
            return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
          };
          f32x2 y = mul2(ff, two(r[c]));
          a[c] = bf16x2(y);
          y = fma2(minus, two(a[c]), y);
          b[c] = bf16x2(y);
          d[c] = bf16x2(fma2(minus, two(b[c]), y));
        }
        to[e] = make_uint4(a[0], a[1], a[2], a[3]);
        to[e + M::kBox / 16] = make_uint4(b[0], b[1], b[2], b[3]);
        to[e + 2 * M::kBox / 16] = make_uint4(d[0], d[1], d[2], d[3]);
      }
      return true;
    };
    // the state as an operand; and V' and it are ready for chunk g
    auto hand_over = [&](uint32_t g) {
      if (OUT && mine)
#pragma unroll
        for (int j = 0; j < 16; j += 8)
          kda_tc::st16(smem + M::kS + kda_tc::mn_off(c0 + j, i, 1024), bf16x2(S[j / 2]),
                       bf16x2(S[j / 2 + 1]), bf16x2(S[j / 2 + 2]), bf16x2(S[j / 2 + 3]));
      sm100::fence_async_smem();
      arrive(&bars.ready[g & 1]);
      if (!OUT) arrive(&bars.gate_empty[g & 1]);
    };
    // The full pass begins and ends a chunk by the same code, one chunk apart: chunk g's K^T V' and
    // O (`old`), chunk g + 1's V', operand of S and P (`more`).  The first pass, whose V' and
    // product have two places each, makes V' of chunk g + 1 before it waits for chunk g's product.
    // (the full pass of segments starts while the scan is at work: Q, K, V and the decays were
    // there before the first pass, and the states are what it waits for here)
    if (OUT && p.states) wait_for_kernel_before();
    bool more = enter(), old = false;
    float factor = 0.0f;  // scale * 2^G of this thread's row
    Walk<OUT> ahead(p, order, !OUT);
    for (uint32_t g = ~0u; more || old; ++g) {
      const uint32_t s = g & 1;
      const int64_t at = it.row + t + row;  // this chunk's rows go out last
      const bool live = row < it.len - t;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) +
                                            (at * p.a.H + it.h) * p.a.dv + NV * it.half + c0);
      if (!OUT && ahead.valid) {
        if (!weigh(g + 1)) break;
        hand_over(g + 1);
        ahead.next();
      }
      if (old) {
        if (!wait(&bars.ds_done[g % NS], g / NS)) break;
        sm100::tc_fence_after();
        float x[16], y[16], z[16];
        const uint32_t from = tm + (OUT ? TM_DS : s ? TM_D1 : TM_D0) + c0;
        sm100::tmem_ld16(from, x);
        sm100::tmem_ld16(from + NV, y);
        if (!OUT) sm100::tmem_ld16(from + 2 * NV, z);
        const float4 f = *reinterpret_cast<const float4*>(&totals[g % kTotals]);
        const bool forget = __float_as_int(f.z) < C;
        const f32x2 hi = pair(f.x, f.x), lo = pair(f.y, f.y);
        sm100::tmem_wait_ld();
        sm100::tc_fence_before();
        if (!OUT) {
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] += z[e];
        }
        if (forget) {
#pragma unroll
          for (int e = 0; e < 8; ++e) S[e] = pair(0.0f, 0.0f);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          S[e] = fma2(hi, S[e], fma2(lo, S[e], add2(pair(x[2 * e], x[2 * e + 1]),
                                                    pair(y[2 * e], y[2 * e + 1]))));
        if (!OUT) {
          all *= (double)f.x + (double)f.y;
          gone |= forget;
        }
        t += C;
        if (t >= it.len) {
          leave();
          id = following(id);
          more = enter();
        }
      }
      if (OUT && more) {
        if (!weigh(g + 1)) break;
        hand_over(g + 1);
      }
      uint32_t rows[8];  // O of chunk g, 16 columns
      if (OUT && old) {
        const f32x2 ff = pair(factor, factor), scale = pair(p.a.scale, p.a.scale);
        if (!wait(&bars.o_done[s], g >> 1)) break;
        sm100::tc_fence_after();
        float x[16], y[16];
        sm100::tmem_ld16(tm + TM_O1 + NV * s + c0, x);
        sm100::tmem_ld16(tm + TM_O2 + c0, y);
        sm100::tmem_wait_ld();
        sm100::tc_fence_before();
        const int first = totals[g % kTotals].first;
        if (first < C) {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = row >= first ? 0.0f : x[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          rows[e] = bf16x2(fma2(ff, pair(x[2 * e], x[2 * e + 1]),
                                mul2(scale, pair(y[2 * e], y[2 * e + 1]))));
      }
      if (OUT && more) {
        // P, 16 columns at a time
        if (!wait(&bars.s_done, g + 1)) break;
        sm100::tc_fence_after();
        const Gate& gate = gates[s ^ 1];
        const float own = gate.back[row];
        const int2 e = gate.end[q];
        // (where the difference is of two large numbers, what lies between them has forgotten
        // the row's own token: 2^-14 of the factor at 10 tokens of a block that forget)
        factor = p.a.scale * ex2(fixed(e.x, e.y) - own);
#pragma unroll 1
        for (int b = part; b < 8; b += 4) {
          uint32_t out[8] = {};
          if (b < 2 * q + 2) {
            float x[16];
            f32x2 w[8];
            sm100::tmem_ld16(tm + TM_S + 16 * b, x);
            const bool below = b < 2 * q;  // (of the diagonal's 32 columns)
            const int2 o = gate.end[b >> 1];
            float f = fixed(e.x - o.x, e.y - o.y) - own;
            if (below) f = ex2(f);
            const f32x2 ff = pair(f, f);
            const float4* c = reinterpret_cast<const float4*>((below ? gate.col : gate.back) + 16 * b);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 y = c[j];
              w[2 * j] = pair(y.x, y.y);
              w[2 * j + 1] = pair(y.z, y.w);
            }
            if (below) {
#pragma unroll
              for (int j = 0; j < 8; ++j) w[j] = mul2(ff, w[j]);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                float u, v;
                unpair(add2(ff, w[j]), u, v);
                w[j] = pair(ex2(u), ex2(v));
              }
            }
            sm100::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = mul2(w[j], pair(x[2 * j], x[2 * j + 1]));
            if (!below) {
              // (tokens to come are cleared, not multiplied by 0: they may be anything)
              const int last = row - 16 * b;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                float u, v;
                unpair(w[j], u, v);
                w[j] = pair(2 * j <= last ? u : 0.0f, 2 * j + 1 <= last ? v : 0.0f);
              }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = bf16x2(w[j]);
          }
          tmem_st8(tm + TM_P + 8 * b, out);
        }
        sm100::tmem_wait_st();
        sm100::tc_fence_before();
        arrive(&bars.p_full);
        arrive(&bars.gate_empty[(g + 1) & 1]);
      }
      // (the stores come last: an arrival right behind them would wait for them, some 750 cycles.
      // 32 rows' sectors are what a warp stores: once each, where out is aligned to them)
      if (OUT && old && live) {
        if (whole) {
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst),
                       "r"(rows[0]), "r"(rows[1]), "r"(rows[2]), "r"(rows[3]), "r"(rows[4]),
                       "r"(rows[5]), "r"(rows[6]), "r"(rows[7])
                       : "memory");
        } else {
          dst[0] = make_uint4(rows[0], rows[1], rows[2], rows[3]);
          dst[1] = make_uint4(rows[4], rows[5], rows[6], rows[7]);
        }
      }
      old = more;
    }
  }
  __syncwarp();
  sm100::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *s_abort) report(p.a.status, KDA_ERR_TIMEOUT);
  if (warp == 1) sm100::tmem_dealloc(*s_tmem, kTmemCols);
}

// The states that segments start from: column by column of a sequence,
// S(s) <- gamma(s) S(s - 1) + S(s), and a copy of the initial state in the
// last one's place.
constexpr int kScanThreads = 256;
__global__ void __launch_bounds__(kScanThreads) kda_linear_scan_kernel(const TileArgs p) {
  kernel_may_follow();
  wait_for_kernel_before();
  const int size = p.a.dk * p.a.dv, blocks = size / (4 * kScanThreads);
  const int unit = blockIdx.x / blocks, n = unit / p.a.H, h = unit - n * p.a.H;
  const int e = 4 * ((blockIdx.x - unit * blocks) * kScanThreads + threadIdx.x);
  int64_t row;
  int len;
  if (!span(p.a, n, row, len)) return;
  const int segs = (len + p.seg - 1) / p.seg;
  const int col = p.a.cu ? (int)(row / p.seg) + n : n * p.segs;
  if (segs < 2) return;
  auto at = [&](int s) {
    return reinterpret_cast<float4*>(p.states + ((int64_t)(col + s) * p.a.H + h) * size + e);
  };
  *at(segs - 1) = p.a.init ? *reinterpret_cast<const float4*>(p.a.init + unit * (int64_t)size + e)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
  float4 x = *at(0);
  for (int s0 = 1; s0 < segs - 1; s0 += 8) {  // (their loads together)
    float4 y[8];
    float2 f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s0 + k < segs - 1) {
        y[k] = *at(s0 + k);
        f[k] = p.gammas[(int64_t)(col + s0 + k) * p.a.H + h];
      }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s0 + k < segs - 1) {
        if (f[k].x < 0.0f) x = make_float4(0.f, 0.f, 0.f, 0.f);
        x.x = fmaf(f[k].x, x.x, fmaf(f[k].y, x.x, y[k].x));
        x.y = fmaf(f[k].x, x.y, fmaf(f[k].y, x.y, y[k].y));
        x.z = fmaf(f[k].x, x.z, fmaf(f[k].y, x.z, y[k].z));
        x.w = fmaf(f[k].x, x.w, fmaf(f[k].y, x.w, y[k].w));
        *at(s0 + k) = x;
      }
  }
}

// 3-D map over rows `stride` elements apart of `heads` heads of d channels:
// boxes of 64 channels x 1 head x 128 rows, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int heads, int d, int64_t stride) {
  auto enc = kda_tc::get_encode();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, 1, C};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How the token axis is cut.  Times in chunks of one CTA (1.9 us): segments cost 0.4 of
// their chunks and six more.  Both numbers are what the choices went best with; a chunk of
// the first pass alone takes 0.55 of one of the full pass, but a rule with that number and no
// price for an item of its own takes many short segments: 8192 tokens of 16 heads go from 71 us
// (four segments; 133 whole) to 119 (32).  Cut against whole: 4096 tokens of 4 heads 27
// and 69 us, 32 768 of 4 heads 69 and 492, 131 072 of 16 heads 750 and 1958; 4096 tokens of 32
// heads 72 both ways.  Packed lengths are not known here: the longest is taken for twice the
// mean.  Where they are all alike that is too long (4 sequences of 4096 tokens, 8 heads: cut,
// 130 us; whole they would take 72), where one is much longer too short (32 000 tokens among 31
// sequences of 10, 8 heads: whole, 497 us).
struct Cut {
  int seg, segs, cols;
};
Cut cut(int N, int64_t T, int H, int dv, bool packed) {
  const int sms = kda_device_sms() > 0 ? kda_device_sms() : 148;
  const int64_t units = (int64_t)H * (dv / NV);
  const int64_t longest = packed ? (T < 2 * T / N ? T : 2 * T / N) : T;
  const int64_t chunks = (longest + C - 1) / C;
  auto waves = [&](int64_t items, int64_t each) {  // items of `each` chunks on all SMs
    return (items + sms - 1) / sms * each;
  };
  const int64_t all = packed ? (T + C - 1) / C + N / 2 : chunks * N;  // chunks of a head's columns
  double best = packed ? (double)(all * units / sms > chunks ? all * units / sms : chunks)
                       : (double)waves((int64_t)N * units, chunks);
  int64_t pick = 0;
  for (int64_t segs = 2; segs <= 64 && segs * 2 <= chunks; ++segs) {
    const int64_t each = (chunks + segs - 1) / segs;
    const int64_t items = packed ? ((all + each - 1) / each) * units : N * segs * units;
    const double t = 1.4 * waves(items, each) + 6.0;
    if (t < 0.9 * best) {
      best = t;
      pick = each;
    }
  }
  Cut c;
  c.seg = pick ? (int)(pick * C) : 1 << 30;
  if (!packed)
    c.segs = pick ? (int)((T + c.seg - 1) / c.seg) : 1;
  else
    c.segs = 1;
  c.cols = packed ? (pick ? (int)(T / c.seg) + N : N) : N * c.segs;
  return c;
}

size_t r256(size_t x) { return (x + 255) / 256 * 256; }

template <int DK, bool OUT>
kda_status launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                  const TileArgs& p, cudaStream_t s) {
  auto kernel = kda_linear_tile_kernel<DK, OUT>;
  const kda_status rc = kda_smem_attr((const void*)kernel, Smem<DK, OUT>::kBytes);
  if (rc != KDA_OK) return rc;
  const int64_t items = (int64_t)p.cols * p.a.H * p.halves;  // (below 2^30: N * H is)
  const int sms = kda_device_sms();
  const unsigned grid = (unsigned)(items < sms ? items : sms);
  if (OUT && p.states)
    return launch_following(kernel, grid, kThreads, Smem<DK, OUT>::kBytes, s, q, k, v, p);
  kernel<<<grid, kThreads, Smem<DK, OUT>::kBytes, s>>>(q, k, v, p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <int DK>
kda_status run(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
               const TileArgs& p, cudaStream_t s) {
  if (p.states) {
    kda_status rc = launch<DK, false>(q, k, v, p, s);
    if (rc != KDA_OK) return rc;
    const unsigned grid = (unsigned)(p.a.N * p.a.H * (p.a.dk * p.a.dv / (4 * kScanThreads)));
    rc = launch_following(kda_linear_scan_kernel, grid, kScanThreads, 0, s, p);
    if (rc != KDA_OK) return rc;
  }
  return launch<DK, true>(q, k, v, p, s);
}

}  // namespace

bool kda_linear_tile_ok(int dk, int dv, kda_dtype dtype) {
  return dtype == KDA_BF16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128);
}

size_t kda_linear_tile_workspace(int N, int T, int H, int dk, int dv, bool packed) {
  const Cut c = cut(N, T, H, dv, packed);
  if (c.seg > T) return 0;
  return r256((size_t)c.cols * H * dk * dv * 4) + r256((size_t)c.cols * H * 8);
}

kda_status kda_launch_linear_tile(const LinearArgs& a, void* workspace, cudaStream_t s) {
  const bool packed = a.cu != nullptr;
  const Cut c = cut(a.N, a.T, a.H, a.dv, packed);
  TileArgs p{a, c.seg, c.segs, c.cols, a.dv / NV, nullptr, nullptr};
  if (c.seg <= a.T) {
    p.states = static_cast<float*>(workspace);
    p.gammas = reinterpret_cast<float2*>(static_cast<unsigned char*>(workspace) +
                                         r256((size_t)c.cols * a.H * a.dk * a.dv * 4));
  }
  const int64_t rows = packed ? a.T : (int64_t)a.N * a.T;
  CUtensorMap q, k, v;
  if (!make_map(&q, a.q, rows, a.HK, a.dk, a.q_stride) ||
      !make_map(&k, a.k, rows, a.HK, a.dk, a.k_stride) ||
      !make_map(&v, a.v, rows, a.H, a.dv, a.v_stride))
    return KDA_ERR_CUDA;
  return a.dk == 64 ? run<64>(q, k, v, p, s) : run<128>(q, k, v, p, s);
}
