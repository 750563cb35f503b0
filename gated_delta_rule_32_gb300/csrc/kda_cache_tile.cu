// kda_cache_tile.cu -- attention over the paged cache for requests with more
// than a few query rows per key / value head (prompts, pieces of prompts),
// on the tcgen05 tensor cores.
//
// A pair of CTAs (a cluster of two SMs) works on segments: up to 512 query rows
// of one (request, key / value head) -- rows are (token, head of the group)
// pairs, so the group shares the keys it reads -- against a range of 128-token
// key tiles.  Two row tiles of 256 rows, 128 in each CTA, alternate: while one's
// softmax runs, the tensor cores work for the other.  Each CTA converts and
// holds half of a key tile (64 tokens) and of a value tile (half the channels);
// a product reads both halves (cta_group::2).  With one CTA a tile, shared
// memory was what bound this kernel: its operands, 128 bytes a cycle of the
// scores' products, left none for the other warps' traffic.
// Warps of a CTA:
//   0-3, 4-7   softmax of row tile 0 / 1, one thread per row
//   8-11       keys:   codes -> f16 operand tiles in shared memory
//   12-15      values: the same; between segments 8-15 convert the queries
//   16         owns tensor memory; of the first CTA: issues all products (in
//              step, one thread carrying them out); of the second: tells the
//              first that its keys and queries are there
//   17         walks the schedule and looks up the pages' scales, some key
//              tiles ahead of the softmax
//   18, 19     bring the next segment's queries into L2; of the second CTA 19
//              tells the first that its values are there
// Tensor memory (512 columns): S of both tiles (the weights P replace S in
// place, in f16), O of both tiles.
//
// Codes are exact in f16, so the only roundings of the products' inputs are
// those of P (11 bits, and 2^-25 of the reference's weight and the largest
// value scale at the small end) and of small query elements next to large ones
// of the same row.  A page's key scale multiplies its scores after the product;
// its value scale multiplies its columns of P, relative to a power of two at
// least as large (vref), which leaves O at the end.
//
// Bound by the products where rows are many: 4 D flops for each row and token,
// at 2048 tokens on 32768 cached (32 heads on 4, d = 128, e4m3) 827 us, 1371 TFLOP/s;
// the tensor cores work 2 x 1024 of the 2.6-2.9k cycles that a key tile of both
// row tiles takes, and the rest is the chain of one row tile, which the other's
// products cover in part only: products 1024 -> softmax 1480-1900 (exponentials
// at 32 a cycle an SM) -> store and arrivals about 420.  Measured against it:
// one CTA a tile 1026 us; S in two halves, so that a row tile's products and
// softmax overlap, 914-1040 us (products of 64 tokens take 48 cycles, not 32:
// shared memory); a second warp issuing products 950-987 us.  Prompts without a
// cache, 9 of up to 4096 tokens (32 heads on 8): int8 475 us, 898 TFLOP/s, e4m3 458;
// half of a tile on the diagonal is masked, and a segment's own cost (queries in, O
// out) weighs more where its keys are few.
#include <type_traits>

#include "kda_cache_attn.cuh"
#include "sm100.cuh"

namespace {

using namespace kda_cache;

// Five warpgroups launched with 96 registers a thread; they share them out
// anew (setmaxnreg): 2 x 152 + 2 x 64 + 48 = 5 x 96.  Prompts of up to 4096
// tokens and 2048 tokens on 32768 cached took 466 and 842 us so, 502 and 878
// with 136 / 72 / 64, 481 and 880 with 144 / 72 / 48, 479 and 894 with
// 160 / 56 / 48, where the converters spill in their loop.  (At d = 128 84 to 88
// bytes a thread are spilled all the same, at d = 64 none without pieces.)
constexpr int kThreads = 640;
constexpr int kRegsSoftmax = 152, kRegsConvert = 64, kRegsIssue = 48;
static_assert(2 * kRegsSoftmax + 2 * kRegsConvert + kRegsIssue == 5 * 96, "registers at launch");
constexpr int kTok = 128;    // tokens per key tile
// A worker takes a longer run of key tiles in pieces, O and the sums of weights
// starting anew in each and put together in fp32: a product's addition to O loses
// 2^-24 of it on the average, always towards zero, so that a million tokens with
// values of one sign came out 0.7% too small.  The 65536 tokens of a piece lose 2^-12.
// Only where the table has room for more tokens than that is the form with pieces
// launched: 2048 tokens on 32768 cached take 867 us with it, 828 without (d = 128,
// e4m3; int8 845 and 851, prompts 479 and 477): the code's size and layout.
constexpr int kPiece = 512;
constexpr uint64_t kWaitNs = 2000000000ull;

// Key and value tiles in shared memory: what 227 KB hold beside the queries at
// D = 128.
constexpr int kStages = 4;

template <int D>
struct Smem {
  static constexpr int kQTile = 128 * D * 2;         // a row tile's queries
  static constexpr int kTile = 64 * D * 2;           // this CTA's half of a key or value tile
  static constexpr int kQ = 0;                       // 2 tiles
  static constexpr int kK = 2 * kQTile;              // kStages
  static constexpr int kV = kK + kStages * kTile;    // kStages
  static constexpr int kStage = kV + kStages * kTile;  // 64 bytes of 32 rows for each softmax warp
  static constexpr int kStageRow = 80;               // (a row's 64 bytes, padded against conflicts)
  static constexpr int kStageWarp = 32 * kStageRow;
  static constexpr int kBytes = kStage + 8 * kStageWarp + 1024;
};

// "leader": only the first CTA's is used, both arrive there.  "operands": each
// CTA's own, of its converting warps, and the first's has one arrival more, by
// which the second CTA says that its half is there too.  The others are each
// CTA's own; those that products complete are completed in both.
struct Bars {
  uint64_t q_full[2][2];              // operands; row tile, and parity of its segments
  uint64_t qs_full[2][2], q_empty[2];
  uint64_t s_full[2], o_full[2];
  uint64_t p_full[2];                 // leader
  uint64_t k_full[kStages], v_full[kStages];  // operands
  uint64_t k_empty[kStages], v_empty[kStages];
  uint64_t seg_full[2], seg_empty[2];
  uint64_t sc_full[4], sc_empty[4];
  uint64_t drain;
};

// A segment as the schedule's warp hands it to the others; rows = 0 ends.
struct Seg {
  int r, h, c0, n, kv;     // request and head
  int tok0, rows;          // first token of the row tile in the request, query rows
  int b0, b1, w0, w1, nu;  // key tiles [b0, b1), a piece of the worker's [w0, w1), of nu
};
constexpr int kReaders = 19;  // warps that read it

// The scales of a key tile: of tokens 16 i .. 16 i + 15, the factor from a
// product of codes to log2 units (without the query row's) and the value
// scale, and the largest value scale.
struct Scales {
  float2 k[4], v[4];
  float vmax;
};
constexpr int kRing = 4;

// Bounded wait that also gives up when another warp of the CTA has.  The hint
// lets the hardware suspend the warp for up to 1 ms at a time: a warp that
// polls takes issue slots from the one that issues the products.  What is waited
// for: of threads of this CTA (kOwn); of the pair or its products, after which
// shared memory is written or handed to products (kPair); or tensor memory alone,
// which the fences of tcgen05 order on both sides, so that the barrier has only to
// order the execution (kTensor).
enum Of { kOwn, kPair, kTensor };
template <Of OF = kOwn>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  auto poll = [&]() -> bool {
    uint32_t ok;
    const uint32_t at = sm100::smem_u32(bar), hint = 1000000;
    if (OF == kOwn)
      asm volatile(
          "{\n .reg .pred p;\n"
          " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
          " selp.u32 %0, 1, 0, p;\n}"
          : "=r"(ok) : "r"(at), "r"(parity), "r"(hint) : "memory");
    else if (OF == kPair)
      asm volatile(
          "{\n .reg .pred p;\n"
          " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
          " selp.u32 %0, 1, 0, p;\n}"
          : "=r"(ok) : "r"(at), "r"(parity), "r"(hint) : "memory");
    else
      asm volatile(
          "{\n .reg .pred p;\n"
          " mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
          " selp.u32 %0, 1, 0, p;\n}"
          : "=r"(ok) : "r"(at), "r"(parity), "r"(hint) : "memory");
    return ok != 0;
  };
  if (poll()) return true;
  const uint64_t t0 = sm100::globaltimer_ns();
  for (;;) {
    if (poll()) return true;
    if (*abort) return false;
    if (sm100::globaltimer_ns() - t0 > kWaitNs) {
      *abort = 1;
      return false;
    }
  }
}

// Arrives at the first CTA's copy of a barrier: with what this thread has seen
// and written before, or (tensor memory, after tcgen05's fence) without.  A
// release to the cluster waits for the thread's own accesses under way, 1000
// cycles in a warp that fetches codes, so warps that have none do it for all:
// 2048 tokens on 32768 cached took 1049 us with a release by each converting
// warp (before later steps), 907 with both kinds of operands told by one warp, 826 by two.
__device__ __forceinline__ void arrive_leader_release(uint64_t* bar) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n"
      " mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n}" ::"r"(sm100::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void arrive_leader_tensor(uint64_t* bar) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n"
      " mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n}" ::"r"(sm100::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void tmem_ld32(uint32_t ta, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(ta));
}

// Waits for this thread's loads; the registers pass through it, so that no
// use of them is moved before it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                 "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t ta, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(ta),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Pairs of fp32 values in one 64-bit register, two results an instruction.
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
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
// The products, issued by a whole warp that runs in step, of which one thread
// (`one`) carries them out; four k-steps an asm block.  Issue slots are what
// this warp must not lack, its scheduler serving four busy warps beside it: in
// a branch of one thread the operands are not known to be uniform, and a
// 128 x 128 x 16 product took 97-105 cycles to issue; in step it takes the
// tensor cores' own 64.  With the other warps issuing all the time it took
// 141 with 64-bit descriptor arithmetic for each product, 100 in this form.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(r));
  return r;
}
// D (+)= A B^T, A and B in shared memory, [chunk][row][16 bytes] with 128 and 64
// rows: the low words of their descriptors go up by two chunks a k-step.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t a_hi,
                                        uint32_t b_hi, uint32_t idesc, uint32_t accumulate,
                                        uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b64 a, b;\n .reg .b32 x, y;\n"
      " setp.ne.b32 q, %7, 0;\n setp.ne.b32 p, %6, 0;\n setp.eq.b32 t, 0, 0;\n"
      " mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %4};\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n"
      " add.u32 x, %1, 256;\n add.u32 y, %2, 128;\n mov.b64 a, {x, %3};\n mov.b64 b, {y, %4};\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n"
      " add.u32 x, %1, 512;\n add.u32 y, %2, 256;\n mov.b64 a, {x, %3};\n mov.b64 b, {y, %4};\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n"
      " add.u32 x, %1, 768;\n add.u32 y, %2, 384;\n mov.b64 a, {x, %3};\n mov.b64 b, {y, %4};\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
// The same with A in tensor memory, 8 columns a k-step, and B's rows the
// contracted index: 16 of them a k-step.
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                        uint32_t idesc, uint32_t accumulate, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b64 b;\n .reg .b32 x, y;\n"
      " setp.ne.b32 q, %6, 0;\n setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, 0, 0;\n"
      " mov.b64 b, {%2, %3};\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %4, p;\n"
      " add.u32 x, %1, 8;\n add.u32 y, %2, 16;\n mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], [x], b, %4, t;\n"
      " add.u32 x, %1, 16;\n add.u32 y, %2, 32;\n mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], [x], b, %4, t;\n"
      " add.u32 x, %1, 24;\n add.u32 y, %2, 48;\n mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], [x], b, %4, t;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
// Arrives at a barrier of both CTAs when the products so far are done.
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint32_t one) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q tcgen05.commit.cta_group::2.mbarrier::"
      "arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n}" ::"r"(sm100::smem_u32(bar)),
      "r"(one), "h"((uint16_t)3)
      : "memory");
}

// f(0), ..., f(N - 1), the argument a constant
template <int N, int I = 0, class F>
__device__ __forceinline__ void for_each_of(F f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    for_each_of<N, I + 1>(f);
  }
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Instruction descriptor, f16 operands and fp32 accumulation (the formats of
// A and B are 0).
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// sum_{i < n} floor((a i + b) / 128), n < 2^24: the lattice points under a
// line, by the steps of Euclid's algorithm (Graham, Knuth and Patashnik,
// Concrete Mathematics, section 3.5); a is below 128 after the first step, so
// everything but the sum fits 32 bits.
__device__ inline int64_t sum_tiles(uint32_t n, uint32_t a, uint32_t b) {
  int64_t sum = (int64_t)n * (n - 1) / 2 * (a >> 7) + (int64_t)n * (b >> 7);
  if (n == 0) return 0;
  uint32_t m = 128;
  a &= 127;
  b &= 127;
  for (;;) {
    const uint32_t y = a * n + b;
    if (y < m) return sum;
    n = y / m;
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
    sum += (int64_t)n * (n - 1) / 2 * (a / m) + (int64_t)n * (b / m);
    a %= m;
    b %= m;
  }
}

// What a segment costs beside its key tiles (queries in, O out, the first
// tile's maximum), in key tiles: the schedule counts it as so many units that
// hold no work.  Prompts of up to 4096 tokens took 531 / 505 / 501 / 528 us with
// 2 / 3 / 4 / 6 of them.
constexpr int kLead = 4;

// The row tiles of a request: tile i holds tokens [i tt, (i + 1) tt) and sees
// the first `seen(i)` tokens, in key tiles of which it has one at least.
struct Tiles {
  int n, kv, tt, count;
  __device__ Tiles(const Req& q, const AttnArgs& p) : n(q.n), kv(q.kv), tt(kTileRows / p.G) {
    count = q.n * (int64_t)p.G > p.few_max ? (q.n + tt - 1) / tt : 0;
  }
  __device__ int seen(int i) const { return max(0, kv - n + min(n, (i + 1) * tt)); }
  __device__ int keys(int i) const { return max(1, (int)(((uint32_t)seen(i) + kTok - 1) / kTok)); }
  // units of the tiles before i
  __device__ int64_t before(int i) const {
    const int last = min(i, count - 1);  // the full tiles among them
    const int first = kv - n + tt;       // what a full tile 0 sees
    // tiles that see at most one key tile
    int few = first > kTok ? 0 : (int)((uint32_t)(kTok - first) / (uint32_t)tt) + 1;
    few = few < last ? few : last;
    int64_t s = (int64_t)kLead * i + few +
                sum_tiles(last - few, tt, (uint32_t)first + (uint32_t)few * tt + kTok - 1);
    if (i > last) s += keys(last);
    return s;
  }
};

// Walks a CTA's share, segment by segment: key tiles [b0, b1) of nu.
struct Walk {
  const AttnArgs& p;
  int64_t u, u1, base;  // next unit, end of the share, units before request r
  int r, h, tile, b0, b1, nu;
  int64_t per_head, seg0;  // units of a head, units before the segment
  Req q;
  Tiles t;
  // (a whole warp, every lane with the same values)
  __device__ Walk(const AttnArgs& p_, const Share& s)
      : p(p_), u(s.u0), u1(s.u1), base(s.base), r(s.r), h(0), tile(0), b0(0), b1(0), nu(0),
        per_head(0), seg0(0), q{0, 0, 0}, t(Req{0, 0, 0}, p_) {
    if (u >= u1) return;
    load();
    const int64_t in = u - base;
    h = (int)quotient(in, per_head);
    const int64_t left = in - h * per_head;
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {  // the last tile with at most `left` units before it
      const int step = (hi - lo + 31) >> 5, mid = lo + step * (threadIdx.x & 31);
      const uint32_t yes = __ballot_sync(~0u, mid < hi && t.before(min(mid, t.count)) <= left);
      lo += step * (31 - __clz(yes));
      hi = min(hi, lo + step);
    }
    tile = lo;
    seg0 = base + h * per_head + t.before(tile);
    set();
    if (b0 == b1) next();
  }
  __device__ void load() {
    bool bad;
    q = load_req(p, r, bad);
    t = Tiles(q, p);
    per_head = t.count ? t.before(t.count) : 0;
  }
  __device__ void set() {
    nu = t.keys(tile);
    b0 = max(0, (int)(u - seg0) - kLead);
    b1 = max(0, (int)min((int64_t)nu, u1 - seg0 - kLead));
  }
  __device__ bool live() const { return u < u1; }
  __device__ void next() {
    do {
      seg0 += kLead + nu;
      u = seg0;
      if (u >= u1) return;
      if (++tile == t.count) {
        tile = 0;
        if (++h == p.Hkv) {
          h = 0;
          base += per_head * p.Hkv;
          do {
            ++r;
            load();
          } while (t.count == 0);
        }
      }
      set();
    } while (b0 == b1);
  }
  __device__ int tokens() const { return min(t.tt, q.n - tile * t.tt); }
};

template <int CODE, int D, bool PIECES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    kda_cache_attn_tile_kernel(AttnArgs p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ Bars bars;
  __shared__ Seg s_seg[2];
  __shared__ Scales s_scales[kRing];
  __shared__ float s_qscale[2][256];  // what a query row was divided by
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  unsigned char* smem = smem_raw + ((1024u - (sm100::smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lg = p.page_log2, P = 1 << lg;
  volatile int* abort = &s_abort;
  const int rank = cluster_rank(), pair = blockIdx.x >> 1;

  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     sm100::smem_u32(&s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < 2; ++i) {
      for (int x = 0; x < 2; ++x) {
        sm100::mbar_init(&bars.q_full[i][x], 8 + (rank == 0));  // (a warp's arrival is one)
        sm100::mbar_init(&bars.qs_full[i][x], 8);
      }
      sm100::mbar_init(&bars.q_empty[i], 1);
      sm100::mbar_init(&bars.s_full[i], 1);
      sm100::mbar_init(&bars.o_full[i], 1);
      sm100::mbar_init(&bars.p_full[i], 8);
      sm100::mbar_init(&bars.seg_full[i], 1);
      sm100::mbar_init(&bars.seg_empty[i], kReaders);
    }
    for (int i = 0; i < kStages; ++i) {
      sm100::mbar_init(&bars.k_full[i], 4 + (rank == 0));
      sm100::mbar_init(&bars.v_full[i], 4 + (rank == 0));
      sm100::mbar_init(&bars.k_empty[i], 1);
      sm100::mbar_init(&bars.v_empty[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      sm100::mbar_init(&bars.sc_full[i], 1);
      sm100::mbar_init(&bars.sc_empty[i], 8);
    }
    sm100::mbar_init(&bars.drain, 1);
    sm100::fence_mbar_init();
  }
  sm100::tc_fence_before();
  kernel_may_follow();
  const Share share = find_share<kThreads>(p, pair, [&](const Req& q) {
    const Tiles t(q, p);
    return t.count ? t.before(t.count) * p.Hkv : 0;
  });
  cluster_sync();  // (both CTAs' barriers are there)
  sm100::tc_fence_after();
  constexpr uint32_t tmem = 0;  // (all 512 columns are this CTA's)
  uint32_t nseg = 0;  // segments seen
  // a wait of a whole warp; the next segment, or rows = 0 at the end (or when a
  // wait gave up)
  auto all_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(~0u, wait(bar, parity, abort));
  };
  auto pair_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(~0u, wait<kPair>(bar, parity, abort));
  };
  auto tensor_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(~0u, wait<kTensor>(bar, parity, abort));
  };
  auto next_seg = [&]() -> Seg {
    const uint32_t slot = nseg & 1;
    Seg g;
    if (all_wait(&bars.seg_full[slot], (nseg >> 1) & 1)) {
      g = s_seg[slot];
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&bars.seg_empty[slot]);
      ++nseg;
    } else {
      g.rows = 0;
    }
    return g;
  };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    regs_up<kRegsSoftmax>();
    const int wg = warp >> 2, row = 256 * wg + 128 * rank + 32 * (warp & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lanes + 128 * wg, tO = tmem + lanes + 256 + D * wg;
    // A row of a later piece is added to the sum of the pieces before, or ends it.
    auto put_together = [&](const Seg& g, int64_t sum, int64_t piece, int64_t out_row, float m,
                            float l) {
      float2* ml = reinterpret_cast<float2*>(p.parts.ml) + sum;
      const float ma = l == 0.0f ? -INFINITY : m, mb = ml->x, top = fmaxf(ma, mb);
      const float mn = top == -INFINITY ? 0.0f : top;
      float fa = ex2(ma - mn), fb = ex2(mb - mn);
      l = l * fa + ml->y * fb;
      const bool end = g.w0 == 0 && g.b1 == g.nu;
      if (end) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        fa *= inv;
        fb *= inv;
        if (p.lse) p.lse[out_row] = l == 0.0f ? -INFINITY : (mn + log2f(l)) * 0.6931471805599453f;
      } else {
        *ml = make_float2(top, l);
      }
      float4* so = reinterpret_cast<float4*>(p.parts.o + sum * D);
      const float4* po = reinterpret_cast<const float4*>(p.parts.o + piece * D);
#pragma unroll 2
      for (int c = 0; c < D / 4; ++c) {
        const float4 a = po[c], b = so[c];
        const float4 x = make_float4(a.x * fa + b.x * fb, a.y * fa + b.y * fb, a.z * fa + b.z * fb,
                                     a.w * fa + b.w * fb);
        if (end)
          reinterpret_cast<uint2*>(p.out + out_row * D)[c] =
              make_uint2(sm100::pack_bf16x2(x.x, x.y), sm100::pack_bf16x2(x.z, x.w));
        else
          so[c] = x;
      }
    };
    uint32_t seg = 0, it = 0;  // segments and key tiles that this row tile has had
    uint32_t tiles = 0;        // key tiles of every segment
    for (;;) {
      const Seg g = next_seg();
      if (g.rows == 0) break;
      const int nk = g.b1 - g.b0;
      if (256 * wg >= g.rows) {  // (no rows here: only the scales pass by)
        bool ok = true;
        for (int k = 0; ok && k < nk; ++k, ++tiles) {
          ok = all_wait(&bars.sc_full[tiles % kRing], (tiles / kRing) & 1);
          if (ok && lane == 0) sm100::mbar_arrive(&bars.sc_empty[tiles % kRing]);
        }
        if (!ok) break;
        continue;
      }
      const int kv = g.kv, tok = g.tok0 + row / p.G;
      const bool mine = row < g.rows;
      // tokens this row sees, and the fewest and most that a row of the warp does
      int lim = mine ? kv - g.n + tok + 1 : 0;
      const int lim_hi = __reduce_max_sync(~0u, lim);
      if (!mine) lim = lim_hi;
      const int lim_lo = __reduce_min_sync(~0u, lim);
      float m = -INFINITY, l = 0.0f;
      // 1 / vref, a power of two not below the value scales seen; the warp's vref
      float vrel = 0x1p126f, vtop = 0.0f;
      bool ok = all_wait(&bars.qs_full[wg][seg & 1], (seg >> 1) & 1);
      const float qs = s_qscale[seg & 1][128 * wg + 32 * (warp & 3) + lane];
      for (int k = 0; ok && k < nk; ++k, ++it, ++tiles) {
        const Scales& sc = s_scales[tiles % kRing];
        const int t0 = (g.b0 + k) * kTok;
        ok = all_wait(&bars.sc_full[tiles % kRing], (tiles / kRing) & 1);
        if (!ok) break;
        const float vmax = sc.vmax;
        ok = tensor_wait(&bars.s_full[wg], it & 1);
        if (!ok) break;
        sm100::tc_fence_after();
        // Weights with the reference m of the tiles before, in the first tile
        // with the maximum over its first 32 tokens.  Only where a row's
        // weights sum to more than f16 holds, or when a page's value scale passes
        // those before, is the tile's maximum sought, O rescaled and the tile's
        // weights made again.  So S is read once, and O almost never.  (vtop is
        // the warp's: it equals 1 / vrel of the rows that have seen all pages so
        // far, and the others see nothing any more.)
        uint32_t z[64];
        float lt;
        int fresh = k == 0 ? 32 : vmax > vtop ? kTok : 0;  // tokens of the maximum that is sought
        for (;;) {
          if (fresh) {  // (rare: kept short, the loop's code must fit the caches)
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const int c0 = t0 + 32 * c;
              if (c0 >= lim_hi || 32 * c >= fresh) break;
              const float2 ks = sc.k[c];
              uint32_t s[32];
              tmem_ld32(tS + 32 * c, s);
              tmem_wait_ld32(s);
              float a = -INFINITY, b = -INFINITY;
              if (c0 + 32 <= lim_lo) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  a = fmaxf(a, __uint_as_float(s[e]));
                  b = fmaxf(b, __uint_as_float(s[16 + e]));
                }
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  if (c0 + e < lim) a = fmaxf(a, __uint_as_float(s[e]));
                  if (c0 + 16 + e < lim) b = fmaxf(b, __uint_as_float(s[16 + e]));
                }
              }
              // (a group of which the row sees nothing: its scale may be 0)
              if (c0 < lim) mx = fmaxf(mx, a * (ks.x * qs));
              if (c0 + 16 < lim) mx = fmaxf(mx, b * (ks.y * qs));
            }
            // (a row that sees nothing here sees nothing further on: 0 serves)
            const float mn = fmaxf(m, mx) == -INFINITY ? 0.0f : fmaxf(m, mx);
            float f = k == 0 ? 0.0f : ex2(m - mn);
            m = mn;
            l *= f;
            float vm = vmax;  // the largest value scale that the row sees
            if (t0 + kTok > lim_lo) {
              vm = 0.0f;
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                if (t0 + 32 * c < lim) vm = fmaxf(vm, sc.v[c].x);
                if (t0 + 32 * c + 16 < lim) vm = fmaxf(vm, sc.v[c].y);
              }
            }
            if (vm * vrel > 1.0f) {
              const float vnew = pow2_inverse(pow2_above(vm));
              f = f * pow2_inverse(vrel) * vnew;
              vrel = vnew;
            }
            if (vmax > vtop) vtop = pow2_above(vmax);
            if (k > 0) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(tO + 32 * c, o);
                tmem_wait_ld32(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(tO + 32 * c, o);
              }
            }
          }
          f32x2 l2 = pack2(0.0f, 0.0f), m2 = pack2(-m, -m);
          if (t0 + kTok <= lim_lo) {  // every row of the warp sees the whole tile
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float2 ks = sc.k[c], vs = sc.v[c];
              uint32_t s[32];
              tmem_ld32(tS + 32 * c, s);
              const float f0 = ks.x * qs, f1 = ks.y * qs;
              const float v0 = vs.x * vrel, v1 = vs.y * vrel;
              tmem_wait_ld32(s);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float f = e < 16 ? f0 : f1, v = e < 16 ? v0 : v1;
                float a, b;
                unpack2(fma2(pack2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), pack2(f, f),
                             m2), a, b);
                const f32x2 w = pack2(ex2(a), ex2(b));
                l2 = add2(l2, w);
                unpack2(mul2(w, pack2(v, v)), a, b);
                z[16 * c + e / 2] = pack_half(a, b);
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int c0 = t0 + 32 * c;
              if (c0 >= lim_hi) {  // no row of the warp sees these 32 tokens
#pragma unroll
                for (int e = 0; e < 16; ++e) z[16 * c + e] = 0;
                continue;
              }
              const float2 ks = sc.k[c], vs = sc.v[c];
              uint32_t s[32];
              tmem_ld32(tS + 32 * c, s);
              const float f0 = ks.x * qs, f1 = ks.y * qs;
              // (where the row sees nothing of a group its scale may be a NaN)
              const float v0 = c0 < lim ? vs.x * vrel : 0.0f;
              const float v1 = c0 + 16 < lim ? vs.y * vrel : 0.0f;
              tmem_wait_ld32(s);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float f = e < 16 ? f0 : f1, v = e < 16 ? v0 : v1;
                float a = fmaf(__uint_as_float(s[e]), f, -m);
                float b = fmaf(__uint_as_float(s[e + 1]), f, -m);
                if (c0 + e >= lim) a = -INFINITY;
                if (c0 + e + 1 >= lim) b = -INFINITY;
                const f32x2 w = pack2(ex2(a), ex2(b));
                l2 = add2(l2, w);
                unpack2(mul2(w, pack2(v, v)), a, b);
                z[16 * c + e / 2] = pack_half(a, b);
              }
            }
          }
          float la, lb;
          unpack2(l2, la, lb);
          lt = la + lb;
          // no weight above the sum; an infinity or NaN is seen too
          const bool over = !(lt <= kMaxWeights);
          if (fresh == kTok || !__any_sync(~0u, over)) break;
          fresh = kTok;
        }
        l += lt;
        __syncwarp();
        tmem_st32(tS, z);
        tmem_st32(tS + 32, z + 32);
        sm100::tmem_wait_st();
        sm100::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_leader_tensor(&bars.p_full[wg]);
          sm100::mbar_arrive(&bars.sc_empty[tiles % kRing]);
        }
      }
      if (!ok || !tensor_wait(&bars.o_full[wg], seg & 1)) break;
      ++seg;
      sm100::tc_fence_after();
      // (a piece after the first goes to the pair's third slot, and from there to the sum)
      const bool later = PIECES && g.b0 > g.w0, whole = g.b0 == 0 && g.b1 == g.nu;
      const int64_t sum_slot = 2 * (int64_t)pair + ((PIECES ? g.w0 : g.b0) > 0 ? 0 : 1);
      const int64_t slot = later ? 2 * (int64_t)p.parts.ctas + pair : sum_slot;
      const int64_t at = (int64_t)(g.c0 + tok) * p.Hq + g.h * p.G + row % p.G;
      const float ov = pow2_inverse(vrel) * (1.0f / code_top(CODE));
      const float f = whole ? (l == 0.0f ? 0.0f : ov / l) : ov;
      // O leaves through 64-byte row pieces in shared memory, so that a store
      // writes 8 rows' whole sectors and not 32 rows' halves.
      unsigned char* dst_row = whole
                                   ? reinterpret_cast<unsigned char*>(p.out + at * D)
                                   : reinterpret_cast<unsigned char*>(
                                         p.parts.o + (slot * kTileRows + row) * D);
      const uint64_t dst_u = mine ? reinterpret_cast<uint64_t>(dst_row) : 0;
      uint64_t dst[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dst[i] = __shfl_sync(~0u, dst_u, 8 * i + (lane >> 2));
        if (dst[i]) dst[i] += 16 * (lane & 3);
      }
      unsigned char* stage = smem + Smem<D>::kStage + warp * Smem<D>::kStageWarp;
      auto put = [&](const uint32_t (&y)[16], int piece) {
        uint4* mine_at = reinterpret_cast<uint4*>(stage + lane * Smem<D>::kStageRow);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mine_at[i] = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(
              stage + (8 * i + (lane >> 2)) * Smem<D>::kStageRow + 16 * (lane & 3));
          if (dst[i]) *reinterpret_cast<uint4*>(dst[i] + 64 * piece) = v;
        }
        __syncwarp();
      };
      // (a row that has seen nothing: its weights are zeros, so is its sum)
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t y[32], z[16];
        __syncwarp();
        tmem_ld32(tO + 32 * c, y);
        tmem_wait_ld32(y);
        if (whole) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            z[e] = sm100::pack_bf16x2(__uint_as_float(y[2 * e]) * f,
                                      __uint_as_float(y[2 * e + 1]) * f);
          put(z, c);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) z[e] = __float_as_uint(__uint_as_float(y[e]) * f);
          put(z, 2 * c);
#pragma unroll
          for (int e = 0; e < 16; ++e) z[e] = __float_as_uint(__uint_as_float(y[16 + e]) * f);
          put(z, 2 * c + 1);
        }
      }
      sm100::tc_fence_before();
      if (mine && later) {
        put_together(g, sum_slot * kTileRows + row, slot * kTileRows + row, at, m, l);
      } else if (mine) {
        if (!whole) {
          p.parts.ml[(slot * kTileRows + row) * 2] = l == 0.0f ? -INFINITY : m;
          p.parts.ml[(slot * kTileRows + row) * 2 + 1] = l;
        } else if (p.lse) {
          p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
      }
    }
  } else if (warp < 16) {
    // ---------------------------------------------- codes -> f16 operands
    regs_down<kRegsConvert>();
    const int wq = warp & 3, t8 = lane & 7, c4 = lane >> 3;
    uint32_t cnt = 0, n0 = 0, n1 = 0;
    bool ok = true;
    // The queries of a segment, 8 rows of each row tile for a warp at a time:
    // a row is divided by a power of two so that it fits f16, its sign carries
    // the sign of the score's scale.
    auto queries = [&](const Seg& g, int t) -> bool {
      constexpr int C = D / 32;  // 16-byte pieces of a row per lane
      const uint32_t i = t ? n1++ : n0++;
#pragma unroll 1
      for (int g8 = warp - 8; g8 < 16; g8 += 8) {
        const int row = 8 * g8 + t8, of = 256 * t + 128 * rank + row;
        const uint16_t* src = p.q + (int64_t)(g.c0 + g.tok0 + of / p.G) * p.q_stride +
                              (int64_t)(g.h * p.G + of % p.G) * D + 8 * c4;
        uint4 y[C];
#pragma unroll
        for (int c = 0; c < C; ++c) y[c] = load16_if<0>(src + 32 * c, of < g.rows);
        if (g8 == warp - 8 && i > 0 && !pair_wait(&bars.q_empty[t], (i - 1) & 1)) return false;
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint32_t a[4] = {y[c].x, y[c].y, y[c].z, y[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            most = max(most, max(a[e] & 0x7fff0000u, (a[e] << 16) & 0x7fff0000u));
        }
        most = max(most, __shfl_xor_sync(~0u, most, 8));
        most = max(most, __shfl_xor_sync(~0u, most, 16));
        const int ex = row_exponent(most);
        const float down = copysignf(exp2i(-ex), p.scale);
        if (c4 == 0) s_qscale[i & 1][128 * t + row] = exp2i(ex);
        unsigned char* d = smem + Smem<D>::kQ + t * Smem<D>::kQTile + row * 16 + c4 * 2048;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint32_t a[4] = {y[c].x, y[c].y, y[c].z, y[c].w};
          uint32_t f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            f[e] = pack_half(__uint_as_float(a[e] << 16) * down,
                             __uint_as_float(a[e] & 0xffff0000u) * down);
          *reinterpret_cast<uint4*>(d + c * 8192) = make_uint4(f[0], f[1], f[2], f[3]);
        }
      }
      sm100::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        sm100::mbar_arrive(&bars.qs_full[t][i & 1]);
        sm100::mbar_arrive(&bars.q_full[t][i & 1]);
      }
      return true;
    };
    auto convert = [&](auto which) {
      constexpr bool V = decltype(which)::value;
      const uint8_t* codes = V ? p.v_codes : p.k_codes;
      uint64_t* full = V ? bars.v_full : bars.k_full;
      uint64_t* empty = V ? bars.v_empty : bars.k_empty;
      // A piece is 16 codes of a token.  Keys: a warp's 16 tokens, whole rows;
      // values: its 32 tokens, half rows.  N pieces a lane: its token (past the
      // warp's first) and byte of the row of piece i, and where its two
      // 16-byte chunks go.
      constexpr int N = D / 32;
      auto token = [&](int i) {
        return !V ? 8 * (i & 1) + t8 : D == 128 ? 8 * i + t8 : 16 * i + 8 * (c4 >> 1) + t8;
      };
      auto byte = [&](int i) {
        return !V ? 64 * (i >> 1) + 16 * c4 : D == 128 ? 64 * rank + 16 * c4
                                                       : 32 * rank + 16 * (c4 & 1);
      };
      auto chunk = [&](int i) {
        return !V ? 8 * (i >> 1) + 2 * c4 : D == 128 ? 2 * c4 : 2 * (c4 & 1);
      };
      const int first = V ? 32 * wq : 64 * rank + 16 * wq;  // token of a key tile
      unsigned char* tiles = smem + (V ? Smem<D>::kV + first * 16 : Smem<D>::kK + 16 * wq * 16);
      constexpr int kChunk = V ? 2048 : 1024;
      while (ok) {
        const Seg sg = next_seg();
        if (sg.rows == 0) break;
        const int nk = sg.b1 - sg.b0, kv = sg.kv;
        const int32_t* table = p.table + (int64_t)sg.r * p.max_pages;
        // A page holds a divisor of a key tile's tokens, so a token's place in
        // its page is the same in every key tile.
        const uint32_t page_bytes = (uint32_t)(p.Hkv << lg) * D;
        auto place_of = [&](int g) {
          const int at = (sg.h << lg) + ((first + 16 * g) & (P - 1)) + token(0);
          return codes + (int64_t)at * D + byte(0);
        };
        const uint8_t* const at_a = place_of(0);
        const uint8_t* const at_b = place_of(V ? 1 : 0);
        // the pages of the warp's tokens 0-15 and (values) 16-31
        auto page_of = [&](int k, int g) -> int {
          const int64_t t0 = (int64_t)(sg.b0 + k) * kTok + first + 16 * g;
          return load_page_if(table + (t0 >> lg), k < nk && t0 < kv);
        };
        uint4 x[N];
        auto fetch = [&](int k, int pa, int pb) {
          const bool in_a = (uint32_t)pa < (uint32_t)p.num_pages;
          const bool in_b = (uint32_t)pb < (uint32_t)p.num_pages;
          const uint8_t* a = at_a + (uint64_t)(uint32_t)pa * page_bytes;
          const uint8_t* b = at_b + (uint64_t)(uint32_t)pb * page_bytes;
          const int left = kv - (sg.b0 + k) * kTok - first - token(0);
          for_each_of<N>([&](auto piece) {
            constexpr int i = decltype(piece)::value;
            constexpr int g = !V ? 0 : D == 128 ? i >> 1 : i;  // which 16 tokens
            constexpr int off = !V         ? 8 * (i & 1) * D + 64 * (i >> 1)
                                : D == 128 ? 8 * (i & 1) * D
                                           : 0;
            // (what a page holds past the request's end may be a NaN)
            x[i] = load16_if<off>(g ? b : a,
                                  (g ? in_b : in_a) && (!V || token(i) - token(0) < left));
          });
        };
        auto place = [&]() -> bool {  // x -> the next stage
          const int st = cnt % kStages;
          if (cnt >= kStages && !pair_wait(&empty[st], (cnt / kStages - 1) & 1)) return false;
          unsigned char* dst = tiles + st * Smem<D>::kTile;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const uint32_t y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) codes_to_half<CODE>(y[e], f[2 * e], f[2 * e + 1]);
            unsigned char* d = dst + token(i) * 16 + chunk(i) * kChunk;
            *reinterpret_cast<uint4*>(d) = make_uint4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<uint4*>(d + kChunk) = make_uint4(f[4], f[5], f[6], f[7]);
          }
          return true;
        };
        auto placed = [&]() {
          sm100::fence_async_smem();
          __syncwarp();
          if (lane == 0) sm100::mbar_arrive(&full[cnt % kStages]);
          ++cnt;
        };
        fetch(0, page_of(0, 0), V ? page_of(0, 1) : -1);
        ok = place();
        if (!ok) break;
        placed();
        // (the queries while no codes are held in registers)
        ok = queries(sg, 0) && (sg.rows <= 256 || queries(sg, 1));
        if (!ok || nk == 1) continue;
        fetch(1, page_of(1, 0), V ? page_of(1, 1) : -1);
        int pa = page_of(2, 0), pb = V ? page_of(2, 1) : -1;
        for (int k = 1; k < nk; ++k) {
          ok = place();
          if (!ok) break;
          if (k + 1 < nk) fetch(k + 1, pa, pb);
          pa = page_of(k + 2, 0);
          pb = V ? page_of(k + 2, 1) : -1;
          placed();
        }
      }
    };
    // Both operands are laid out [8-channel chunk][token][16 bytes]: core
    // matrices of 8 tokens x 16 bytes, K-major for the keys (contracted over
    // channels), MN-major for the values (contracted over tokens).  Lanes 8 c
    // .. 8 c + 7 of a warp take the same 16 codes of 8 tokens, so the global
    // reads are whole sectors and the shared writes free of conflicts.
    if (warp < 12)
      convert(std::false_type{});
    else
      convert(std::true_type{});
  } else {
    regs_down<kRegsIssue>();
    // (second CTA) operands that are there: said to the first
    auto tell = [&](uint64_t* bar, uint32_t parity) -> bool {
      if (!all_wait(bar, parity)) return false;
      if (lane == 0) arrive_leader_release(bar);
      return true;
    };
    // the last commits (of k_empty, v_empty) must land before a CTA leaves
    auto drained = [&]() {
      volatile int alone = 0;  // (whatever gave up: the products end)
      wait<kPair>(&bars.drain, 0, &alone);
    };
    if (warp == 17) {
      // ------------------------------------------------ schedule and scales
      const float sm = fabsf(p.scale) * 1.4426950408889634f / code_top(CODE);
      Walk w(p, share);
      if (lane == 0) {
        // what the join of parts needs to know of the segment that this CTA
        // enters in its middle
        PartHead ph{0, 0, 0, 0, 0, 0};
        if (w.live() && w.b0 > 0)
          ph = {w.seg0 + kLead, w.seg0 + kLead + w.nu, w.q.c0 + w.tile * w.t.tt,
                w.tokens() * p.G, w.h, 0};
        p.parts.head[pair] = ph;
      }
      uint32_t tiles = 0;
      bool ok = true;
      int b0 = w.b0;  // the piece [b0, b1) of the worker's key tiles
      for (uint32_t i = 0; ok; ++i) {
        ok = i < 2 || all_wait(&bars.seg_empty[i & 1], ((i >> 1) - 1) & 1);
        if (!ok) break;
        if (!PIECES) b0 = w.b0;
        int b1 = w.b1;
        if (PIECES) {  // (equal ones)
          const int pieces = (w.b1 - b0 + kPiece - 1) / kPiece;
          if (pieces > 1) b1 = b0 + (w.b1 - b0 + pieces - 1) / pieces;
        }
        if (lane == 0) {
          Seg g{};
          if (w.live())
            g = {w.r, w.h, w.q.c0, w.q.n, w.q.kv, w.tile * w.t.tt, w.tokens() * p.G, b0, b1, w.b0,
                 w.b1, w.nu};
          s_seg[i & 1] = g;
          sm100::mbar_arrive(&bars.seg_full[i & 1]);
        }
        if (!w.live()) break;
        // lane i < 8 looks up tokens 16 i .. 16 i + 15, a page a tile ahead
        const int32_t* table = p.table + (int64_t)w.r * p.max_pages;
        auto has = [&](int k) {
          return k < b1 && (int64_t)k * kTok + 16 * (lane & 7) < w.q.kv;
        };
        auto page_of = [&](int k) -> int {
          return load_page_if(table + (((int64_t)k * kTok + 16 * (lane & 7)) >> lg), has(k));
        };
        int pg = page_of(b0);
        for (int k = b0; k < b1; ++k, ++tiles) {
          const bool in = (uint32_t)pg < (uint32_t)p.num_pages;
          if (!in && has(k)) report(p.status, KDA_ERR_BAD_PAGES);
          const float ks = load_scale_if(p.k_scale + (int64_t)pg * p.Hkv + w.h, in);
          const float vs = load_scale_if(p.v_scale + (int64_t)pg * p.Hkv + w.h, in);
          pg = page_of(k + 1);
          const uint32_t e = tiles % kRing;
          ok = tiles < kRing || all_wait(&bars.sc_empty[e], (tiles / kRing - 1) & 1);
          if (!ok) break;
          float vmax = vs;
          vmax = fmaxf(vmax, __shfl_xor_sync(~0u, vmax, 1));
          vmax = fmaxf(vmax, __shfl_xor_sync(~0u, vmax, 2));
          vmax = fmaxf(vmax, __shfl_xor_sync(~0u, vmax, 4));
          if (lane < 8) {
            reinterpret_cast<float*>(s_scales[e].k)[lane] = ks * sm;
            reinterpret_cast<float*>(s_scales[e].v)[lane] = vs;
          }
          if (lane == 0) s_scales[e].vmax = vmax;
          __syncwarp();
          if (lane == 0) sm100::mbar_arrive(&bars.sc_full[e]);
        }
        b0 = b1;
        if (!PIECES || b1 == w.b1) {
          w.next();
          b0 = w.b0;
        }
      }
    } else if (warp >= 18) {
      // -------------- queries ahead into L2; values, told to the first CTA
      uint32_t vc = 0;
      for (bool ok = true; ok;) {
        const Seg g = next_seg();
        if (g.rows == 0) break;
        if (rank != 0 && warp == 19) {
          for (int k = g.b0; ok && k < g.b1; ++k, ++vc)
            ok = tell(&bars.v_full[vc % kStages], (vc / kStages) & 1);
          continue;
        }
        const int step = rank ? 32 : 64;
        for (int e = threadIdx.x - 18 * 32; e < 256 * (D / 64); e += step) {
          const int at = e / (D / 64), row = 256 * (at >> 7) + 128 * rank + (at & 127);
          if (row >= g.rows) continue;
          const uint16_t* src = p.q + (int64_t)(g.c0 + g.tok0 + row / p.G) * p.q_stride +
                                (int64_t)(g.h * p.G + row % p.G) * D + 64 * (e % (D / 64));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
        }
      }
    } else if (rank != 0) {
      // -------------------------------- keys and queries, told to the first CTA
      uint32_t n0 = 0, n1 = 0, kc = 0;
      for (bool ok = true; ok;) {
        const Seg g = next_seg();
        if (g.rows == 0) break;
        ok = tell(&bars.k_full[kc % kStages], (kc / kStages) & 1) &&
             tell(&bars.q_full[0][n0 & 1], (n0 >> 1) & 1);
        ++n0;
        if (ok && g.rows > 256) {
          ok = tell(&bars.q_full[1][n1 & 1], (n1 >> 1) & 1);
          ++n1;
        }
        ++kc;
        for (int k = g.b0 + 1; ok && k < g.b1; ++k, ++kc)
          ok = tell(&bars.k_full[kc % kStages], (kc / kStages) & 1);
      }
      drained();
    } else {
      // ----------------------------------------------------------- products
      const uint32_t id_s = idesc_f16(256, kTok, 0), id_o = idesc_f16(256, D, 1);
      const uint32_t one = elect_one();
      // (a descriptor's address field counts 16-byte units)
      const uint64_t dq = sm100::smem_desc(sm100::smem_u32(smem), 2048, 128);
      const uint64_t dk = sm100::smem_desc(sm100::smem_u32(smem), 1024, 128);
      const uint64_t dv = sm100::smem_desc(sm100::smem_u32(smem), 128, 2048);
      const uint32_t q_lo = (uint32_t)dq + Smem<D>::kQ / 16, k_lo = (uint32_t)dk + Smem<D>::kK / 16;
      const uint32_t v_lo = (uint32_t)dv + Smem<D>::kV / 16;
      const uint32_t q_hi = (uint32_t)(dq >> 32), k_hi = (uint32_t)(dk >> 32);
      const uint32_t v_hi = (uint32_t)(dv >> 32);
      constexpr int kTile16 = Smem<D>::kTile / 16, kQTile16 = Smem<D>::kQTile / 16;
      auto scores = [&](int t, int st, bool last) {  // S_t = Q_t K^T
  #pragma unroll
        for (int s = 0; s < D / 64; ++s)
          mma4_ss(128 * t, q_lo + t * kQTile16 + s * 1024, k_lo + st * kTile16 + s * 512, q_hi,
                  k_hi, id_s, s, one);
        mma_commit(&bars.s_full[t], one);
        if (last) mma_commit(&bars.q_empty[t], one);
      };
      auto values = [&](int t, int st, bool first) {  // O_t (+)= P_t V
  #pragma unroll
        for (int s = 0; s < 2; ++s)
          mma4_ts(256 + D * t, 128 * t + 32 * s, v_lo + st * kTile16 + 64 * s, v_hi, id_o,
                  !first || s > 0, one);
      };
      uint32_t n0 = 0, n1 = 0, t0 = 0, t1 = 0;  // segments and key tiles of the row tiles
      uint32_t kc = 0;                          // key tiles before this one
      bool ok = true;
      for (;;) {
        const Seg g = next_seg();
        if (g.rows == 0) break;
        // (a reduction's result is known to be uniform)
        const bool two = __reduce_max_sync(~0u, g.rows) > 256;
        const int nk = __reduce_max_sync(~0u, g.b1 - g.b0);
        {
          const uint32_t st = kc % kStages;
          ok = pair_wait(&bars.k_full[st], (kc / kStages) & 1) &&
               pair_wait(&bars.q_full[0][n0 & 1], (n0 >> 1) & 1);
          if (!ok) break;
          ++n0;
          sm100::tc_fence_after();
          scores(0, st, nk == 1);
          if (two) {
            ok = pair_wait(&bars.q_full[1][n1 & 1], (n1 >> 1) & 1);
            if (!ok) break;
            ++n1;
            sm100::tc_fence_after();
            scores(1, st, nk == 1);
          }
          mma_commit(&bars.k_empty[st], one);
        }
        // A key tile's weights meet the values, and the next key tile's scores
        // follow as soon as their place is free.  What the next step needs of
        // values and keys is waited for while row tile 1's softmax is awaited (it
        // is there as a rule): a wait takes a few hundred cycles even so.
        auto tiles_there = [&](int k) -> bool {
          const uint32_t at = kc + k;
          return pair_wait(&bars.v_full[at % kStages], (at / kStages) & 1) &&
                 (k + 1 == nk ||
                  pair_wait(&bars.k_full[(at + 1) % kStages], ((at + 1) / kStages) & 1));
        };
        ok = tiles_there(0);
        for (int k = 0; ok && k < nk; ++k) {
          const bool last = k + 1 == nk, before_last = k + 2 == nk;
          const uint32_t st = (kc + k) % kStages, nt = (kc + k + 1) % kStages;
          ok = tensor_wait(&bars.p_full[0], t0++ & 1);
          if (!ok) break;
          sm100::tc_fence_after();
          values(0, st, k == 0);
          if (last) mma_commit(&bars.o_full[0], one);
          else scores(0, nt, before_last);
          if (!last) {
            ok = tiles_there(k + 1);
            if (!ok) break;
          }
          if (two) {
            ok = tensor_wait(&bars.p_full[1], t1++ & 1);
            if (!ok) break;
            sm100::tc_fence_after();
            values(1, st, k == 0);
            if (last) mma_commit(&bars.o_full[1], one);
            else scores(1, nt, before_last);
          }
          mma_commit(&bars.v_empty[st], one);
          if (!last) mma_commit(&bars.k_empty[nt], one);
        }
        kc += nk;
        if (!ok) break;
      }
      mma_commit(&bars.drain, one);
      drained();
    }
  }
  __syncwarp();
  sm100::tc_fence_before();
  cluster_sync();  // (nobody's barriers or tensor memory are used any more)
  if (tid == 0 && s_abort) report(p.status, KDA_ERR_TIMEOUT);
  wait_for_kernel_before();  // (this one needs nothing of it, what follows may)
  if (warp == 16)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(s_tmem) : "memory");
}

template <int CODE, int D, bool PIECES>
kda_status launch_tile(const AttnArgs& p, cudaStream_t s) {
  auto kernel = kda_cache_attn_tile_kernel<CODE, D, PIECES>;
  const kda_status rc = kda_smem_attr((const void*)kernel, Smem<D>::kBytes);
  if (rc != KDA_OK) return rc;
  return launch_following(kernel, 2 * p.parts.ctas, kThreads, Smem<D>::kBytes, s, p);
}

template <int CODE, int D>
kda_status launch_form(const AttnArgs& p, cudaStream_t s) {
  if ((int64_t)p.max_pages << p.page_log2 > (int64_t)kPiece * kTok)
    return launch_tile<CODE, D, true>(p, s);
  return launch_tile<CODE, D, false>(p, s);
}

}  // namespace

kda_status kda_launch_attn_tile(const AttnArgs& p, int d, int code, cudaStream_t s) {
  if (code == KDA_I8)
    return d == 64 ? launch_form<KDA_I8, 64>(p, s) : launch_form<KDA_I8, 128>(p, s);
  return d == 64 ? launch_form<KDA_E4M3, 64>(p, s) : launch_form<KDA_E4M3, 128>(p, s);
}
