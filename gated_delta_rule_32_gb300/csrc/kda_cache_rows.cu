// kda_cache_rows.cu -- attention over the paged cache for requests with few
// query rows per key / value head (decode steps, short drafts), and the join
// of parts.
//
// Bound by the cache's bytes: every code is used for at most 16 query rows
// at a time, 2 * 16 flops per byte (more rows of a request run as groups).
// The work is cut in units of 64 NB tokens of a (request, head, group) and every
// CTA takes an equal share of all units, so ragged batches and single long
// requests fill the chip alike; a segment that crosses a CTA boundary leaves
// parts, which kda_attn_join_kernel joins.
//
// 64 requests' decode step on up to 8192 cached tokens (8 heads, d = 128, 654 MB
// of codes): 140 us with the join, 4.7 TB/s; a kernel that only reads as many
// bytes takes 108-118 us, and the SMs' times for equal shares differ by half.
// Two contexts of up to 262144 tokens (4 heads): 78 us.  One request of 700
// tokens: 12 us, of which the schedule, the chain of one CTA and the join take
// about equal parts.  Three CTAs an SM, as many as the registers allow (168 a
// thread; with 16 rows at d = 128 20 bytes spill).  Against 143 us then, shares
// half as long (six an SM) took 141, four CTAs an SM with NB = 1 142.
//
// Warp w of a CTA takes every fourth run of NB 16-token blocks.  Products run on
// mma.m16n8k16 with the tokens (then the channels) on the 16-row side, which
// leaves 8 columns for query rows: S^T = K Q^T, O^T += V^T P^T.  The order of
// the contracted index is free, so a lane's 16-byte chunk of a key row holds
// its channels of all k-steps (queries are loaded in the same order), and its
// chunks of four value rows its channels of all m-tiles: the codes need no
// change of layout.  They come by asynchronous copies into a ring of each
// warp's own -- eight lanes fetch a whole 128-byte row; in a first form, whose
// lanes fetched what they use themselves, L2 sent every byte twice -- with the
// chunks permuted so that neither side meets bank conflicts.
//
// Codes enter the products as the f16 values that they are (codes_to_half).  int8
// codes as f16 subnormals of c + 128, with the bias taken out of the sums at the
// end, would save two instructions for four codes, but the truncations of the
// accumulators then go with 128 times the sum of the weights and not with the
// output: over 32768 tokens a CTA the error was 2.3% of the output, over 131072
// 18%.  Nor did it save time: 64 decode steps 144.5 us so, 142.6 without, with
// 36 rows a request 181 and 161.
#include <type_traits>

#include "kda_cache_attn.cuh"

namespace {

using namespace kda_cache;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Byte offsets of 16-byte chunk c of token t in a block's keys and values.  A
// quarter of a warp reads the chunks of two tokens of keys, and two chunks of
// every second token of four pairs of values; each set covers all banks.
template <int D>
__device__ __forceinline__ int key_at(int t, int c) {
  return D == 128 ? t * 128 + ((c ^ ((t & 1) << 2)) << 4) : t * 64 + (c << 4);
}
template <int D>
__device__ __forceinline__ int value_at(int t, int c) {
  return D == 128 ? t * 128 + ((c ^ (t & 6)) << 4)
                  : (t ^ ((t >> 1) & 1)) * 64 + ((c ^ ((t >> 1) & 2)) << 4);
}

__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// NT: 8-row tiles of query rows.  NB: 16-token blocks that a warp takes at a
// time: two where the registers allow it, so that one's products overlap the
// other's conversion (drafts of 32 requests, d = 64: 36.5 us, 38.1 with one).
template <int D, int NT>
struct Cfg {
  static constexpr int kBlocks = NT == 1 || D == 64 ? 2 : 1;
  static constexpr int kUnit = 16 * kBlocks * kWarps;      // tokens
  static constexpr int kBlockBytes = 32 * D;               // keys and values of a block
  static constexpr int kStage = kBlocks * kBlockBytes;
  static constexpr int kStages = (D == 128 ? 4 : 8) / kBlocks - (NT == 2 ? 1 : 0);
  static constexpr int kWarpBytes = kStage * kStages;      // 12 or 16 KiB
  // Units after which a worker's sums go to its part in memory and start anew:
  // each product's addition loses 2^-24 of the accumulator on the average, always
  // towards zero; the 32768 tokens that a warp then has lose 2^-13.
  static constexpr int kFold = kWarps * 32768 / kUnit;
};

template <int CODE, int D, int NT>
__global__ void __launch_bounds__(kThreads, kRowsPerSm) kda_cache_attn_rows_kernel(AttnArgs p) {
  using C = Cfg<D, NT>;
  constexpr int KS = D / 16;         // k-steps of K Q^T = m-tiles of V^T P^T
  constexpr int KC = D / 64;         // 16-byte chunks of a key row per lane
  constexpr int VB = D / 8;          // bytes of a value row per lane
  constexpr int ROWS = 8 * NT, NB = C::kBlocks, S = C::kStages;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS];
  __shared__ float2 s_sum[2][ROWS];  // maximum and sum of the pieces before, one after the other
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i8 = lane >> 2, j = lane & 3;
  const int lg = p.page_log2, P = 1 << lg, G = p.G;
  unsigned char* ring = smem + warp * C::kWarpBytes;
  const uint32_t ring_u = (uint32_t)__cvta_generic_to_shared(ring);

  auto blocks_of = [&](const Req& q) -> int64_t {
    if ((int64_t)q.n * G > few_max(D)) return 0;
    return max(1, (int)(((int64_t)q.kv + C::kUnit - 1) / C::kUnit));
  };
  kernel_may_follow();
  auto groups_of = [&](const Req& q) { return (q.n * G + kFewRows - 1) / kFewRows; };
  Share sh = find_share<kThreads>(p, blockIdx.x, [&](const Req& q) {
    const int64_t nb = blocks_of(q);
    return nb ? nb * (p.Hkv * groups_of(q)) : 0;
  });
  int r = sh.r;
  int64_t base = sh.base, u = sh.u0;

  if (tid == 0) p.parts.head[blockIdx.x].rows = 0;
  while (u < sh.u1) {
    bool bad;
    const Req rq = load_req(p, r, bad);
    const int64_t nb = rq.n > 0 ? blocks_of(rq) : 0;
    const int groups = nb ? groups_of(rq) : 0;
    if (u >= base + nb * (p.Hkv * groups)) {
      base += nb * (p.Hkv * groups);
      ++r;
      continue;
    }
    const int hg = (int)quotient(u - base, nb), h = hg / groups;
    const int64_t seg0 = base + hg * nb;              // the (request, head, group)'s units
    // of them this worker's, in pieces of kFold
    const int mine0 = (int)(max(sh.u0, seg0) - seg0), mine1 = (int)(min(sh.u1, seg0 + nb) - seg0);
    const int b0 = (int)(u - seg0), b1 = min(mine1, b0 + C::kFold);
    const int row0 = kFewRows * (hg % groups);
    const int rows = min(kFewRows, rq.n * G - row0), kv = rq.kv;
    if (tid == 0 && mine0 > 0) p.parts.head[blockIdx.x] = {seg0, seg0 + nb, rq.c0, rows, h, row0};

    // queries, in the k order of the keys' chunks; each row scaled to f16
    uint32_t qf[NT][KS][2];
    float qs[NT][2];   // factors of this lane's two columns
    int lim[NT][2];    // tokens that they see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = 8 * nt + i8;
      uint4 x[2 * KC];
      uint32_t most = 0;
#pragma unroll
      for (int c = 0; c < 2 * KC; ++c) {
        x[c] = make_uint4(0, 0, 0, 0);
        if (row < rows) {
          const uint16_t* src = p.q + (int64_t)(rq.c0 + (row0 + row) / G) * p.q_stride +
                                (int64_t)(h * G + (row0 + row) % G) * D + 64 * (c >> 1) + 16 * j +
                                8 * (c & 1);
          x[c] = *reinterpret_cast<const uint4*>(src);
        }
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          most = max(most, max(w[e] & 0x7fff0000u, (w[e] << 16) & 0x7fff0000u));
      }
      most = max(most, __shfl_xor_sync(~0u, most, 1));
      most = max(most, __shfl_xor_sync(~0u, most, 2));
      const int ex = row_exponent(most);
      const float down = exp2i(-ex);
#pragma unroll
      for (int c = 0; c < 2 * KC; ++c) {
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
        // channels 8 (c & 1) .. + 7 of the lane's chunk c / 2: two k-steps
        const int s0 = 4 * (c >> 1) + 2 * (c & 1);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          qf[nt][s0 + (e >> 1)][e & 1] = pack_half(__uint_as_float(w[e] << 16) * down,
                                                   __uint_as_float(w[e] & 0xffff0000u) * down);
      }
      const float up = exp2i(ex);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 8 * nt + 2 * j + c;
        qs[nt][c] = __shfl_sync(~0u, up, (2 * j + c) * 4);
        lim[nt][c] = col < rows ? kv - rq.n + (row0 + col) / G + 1 : 0;
      }
    }
    const int all_see = kv - rq.n + row0 / G + 1;  // tokens that every row sees
    const float sm = p.scale * 1.4426950408889634f / code_top(CODE);

    float o[NT][KS][4], m[NT][2], l[NT][2];
    float vinv[NT][2];  // 1 / vref, a power of two not below the value scales seen
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][s][e] = 0.0f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nt][c] = l[nt][c] = 0.0f;
        vinv[nt][c] = 0x1p126f;
      }
    }

    // this warp's runs of NB blocks: 4 (b0 + i) + warp, i < count
    const int all = (int)(((int64_t)kv + 16 * NB - 1) / (16 * NB));
    const int count = max(0, min(b1, (all - warp + kWarps - 1) / kWarps) - b0);
    const int32_t* table = p.table + (int64_t)r * p.max_pages;
    // pages and scales of 32 blocks at a time, one per lane, a batch ahead
    // (checked when they are used)
    auto token_of = [&](int x) { return ((4 * (b0 + x / NB) + warp) * NB + x % NB) << 4; };
    auto has = [&](int x) { return x < count * NB && token_of(x) < kv; };
    auto page_at = [&](int x) { return load_page_if(table + (token_of(x) >> lg), has(x)); };
    auto checked = [&](int pg, int x) -> int {
      if ((uint32_t)pg < (uint32_t)p.num_pages) return pg;
      if (has(x)) report(p.status, KDA_ERR_BAD_PAGES);
      return 0;
    };
    int pg_cur = checked(page_at(lane), lane), pg_next = page_at(32 + lane);
    float ks_cur = p.k_scale[(int64_t)pg_cur * p.Hkv + h];
    float vs_cur = p.v_scale[(int64_t)pg_cur * p.Hkv + h];
    float ks_next = 0.0f, vs_next = 0.0f;

    // block x of this warp -> its place in the ring (all lanes); in_batch
    // counts from the current batch's start
    const uint32_t page_bytes = (uint32_t)(p.Hkv << lg) * D;
    constexpr int ROWL = D / 16;         // lanes a row
    constexpr int ROWS_I = 32 / ROWL;    // rows an instruction
    const int rl = lane / ROWL, cl = lane % ROWL;
    auto issue = [&](int i, int in_batch, int slot) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int pg =
            __shfl_sync(~0u, in_batch + b < 32 ? pg_cur : pg_next, (in_batch + b) & 31);
        if (has(i * NB + b)) {
          const int t0 = token_of(i * NB + b) & (P - 1);
          const uint64_t at = (uint64_t)(uint32_t)pg * page_bytes + (uint32_t)((h << lg) + t0) * D;
          const uint32_t dst = ring_u + slot * C::kStage + b * C::kBlockBytes;
          const uint8_t* k = p.k_codes + at + lane * 16;
          const uint8_t* v = p.v_codes + at + lane * 16;
#pragma unroll
          for (int e = 0; e < 16 / ROWS_I; ++e)
            copy_async16(dst + key_at<D>(e * ROWS_I + rl, cl), k + e * 512);
#pragma unroll
          for (int e = 0; e < 16 / ROWS_I; ++e)
            copy_async16(dst + 16 * D + value_at<D>(e * ROWS_I + rl, cl), v + e * 512);
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(i, i * NB, i);

    int bi = 0;             // blocks since the batch's start
    int slot = 0, fill = S - 1;  // ring places of this run and of the one that is fetched
    for (int i = 0; i < count; ++i, bi += NB) {
      __syncwarp();  // (the place that is filled next has been read)
      if (bi == 32) {
        bi = 0;
        pg_cur = pg_next;
        ks_cur = ks_next;
        vs_cur = vs_next;
        pg_next = page_at((i * NB + 32) + lane);
      }
      if (bi == 8) {
        pg_next = checked(pg_next, i * NB - 8 + 32 + lane);
        ks_next = p.k_scale[(int64_t)pg_next * p.Hkv + h];
        vs_next = p.v_scale[(int64_t)pg_next * p.Hkv + h];
      }
      issue(i + S - 1, bi + (S - 1) * NB, fill);
      fill = fill + 1 == S ? 0 : fill + 1;
      float kf[NB], vs[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        kf[b] = __shfl_sync(~0u, ks_cur, bi + b) * sm;
        vs[b] = __shfl_sync(~0u, vs_cur, bi + b);
      }
      copy_wait<S - 1>();
      __syncwarp();
      const unsigned char* st = ring + slot * C::kStage;
      slot = slot + 1 == S ? 0 : slot + 1;
      const int tok = token_of(i * NB);
      const bool edge = tok + 16 * NB > all_see;
      float vmax = vs[0];
      if (NB == 2) {
        // (a last run's second block may lie past the end: no page, no copy)
        if (tok + 16 >= kv) vs[NB - 1] = kf[NB - 1] = 0.0f;
        vmax = fmaxf(vmax, vs[NB - 1]);
      }

      // (the tests of single tokens only where a run has tokens to hide)
      auto take = [&](auto at_edge) {
        constexpr bool EDGE = decltype(at_edge)::value;
        // S^T = K Q^T
        float x[NB][NT][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[b][nt][e] = 0.0f;
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const unsigned char* sk = st + b * C::kBlockBytes;
            const uint4 ka = *reinterpret_cast<const uint4*>(sk + key_at<D>(i8, 4 * c + j));
            const uint4 kb = *reinterpret_cast<const uint4*>(sk + key_at<D>(i8 + 8, 4 * c + j));
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              uint32_t a0, a1, a2, a3;
              codes_to_half<CODE>(wa[s], a0, a2);
              codes_to_half<CODE>(wb[s], a1, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(x[b][nt], a0, a1, a2, a3, qf[nt][4 * c + s][0], qf[nt][4 * c + s][1]);
            }
          }
          if (EDGE) {  // tokens i8 and i8 + 8, columns 2 j and 2 j + 1
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (tok + 16 * b + i8 + 8 * (e >> 1) >= lim[nt][e & 1]) x[b][nt][e] = NAN;
          }
        }
        // Weights with the standing reference m of each row, which need not be
        // the maximum: it is sought, with shuffles, only in the first run, when
        // weights sum to more than f16 holds, or when the value scale of a page
        // that the row sees passes vref.  Most runs need one vote.  (A masked
        // score is a NaN until here, a masked weight 0.)
        float w[NB][NT][4], lt[NT][2];
        // the largest value scale that a column's row sees
        auto scales_seen = [&](int nt, int c) {
          if (!EDGE) return vmax;
          const float a = tok < lim[nt][c] ? vs[0] : 0.0f;
          return NB == 2 && tok + 16 < lim[nt][c] ? fmaxf(a, vs[NB - 1]) : a;
        };
        // (rows' scales part only where not all see the same pages)
        bool fresh = i == 0 || (!EDGE && vmax * vinv[0][0] > 1.0f);
        for (;;) {
          if (fresh) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float f[2];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float mx = -INFINITY;  // (fmaxf passes over NaN)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                  mx = fmaxf(mx, fmaxf(x[b][nt][c] * (kf[b] * qs[nt][c]),
                                       x[b][nt][c + 2] * (kf[b] * qs[nt][c])));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
                // (a row that sees nothing in the first run sees nothing at all)
                const float mn = i == 0 ? (mx == -INFINITY ? 0.0f : mx) : fmaxf(m[nt][c], mx);
                f[c] = i == 0 ? 0.0f : ex2(m[nt][c] - mn);
                m[nt][c] = mn;
                l[nt][c] *= f[c];
                const float vm = scales_seen(nt, c);
                if (vm * vinv[nt][c] > 1.0f) {
                  const float vnew = pow2_inverse(pow2_above(vm));
                  f[c] = f[c] * pow2_inverse(vinv[nt][c]) * vnew;
                  vinv[nt][c] = vnew;
                }
              }
#pragma unroll
              for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][s][e] *= f[e & 1];
            }
          }
          bool over = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            lt[nt][0] = lt[nt][1] = 0.0f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                w[b][nt][e] = ex2(fmaf(x[b][nt][e], kf[b] * qs[nt][e & 1], -m[nt][e & 1]));
                if (EDGE && tok + 16 * b + i8 + 8 * (e >> 1) >= lim[nt][e & 1]) w[b][nt][e] = 0.0f;
                lt[nt][e & 1] += w[b][nt][e];
              }
            // (columns without a row see no token; a NaN counts as over)
            over |= !(lt[nt][0] <= kMaxWeights && lt[nt][1] <= kMaxWeights);
            if (EDGE) {
              over |= scales_seen(nt, 0) * vinv[nt][0] > 1.0f;
              over |= scales_seen(nt, 1) * vinv[nt][1] > 1.0f;
            }
          }
          if (fresh || !__any_sync(~0u, over)) break;
          fresh = true;
        }
        uint32_t pb[NB][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          l[nt][0] += lt[nt][0];
          l[nt][1] += lt[nt][1];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[e] = w[b][nt][e] * (vs[b] * (EDGE ? vinv[nt][e & 1] : vinv[0][0]));
              // (0 times a scale that may be NaN)
              if (EDGE && tok + 16 * b + i8 + 8 * (e >> 1) >= lim[nt][e & 1]) y[e] = 0.0f;
            }
            pb[b][nt][0] = transpose8x8(pack_half(y[0], y[1]));
            pb[b][nt][1] = transpose8x8(pack_half(y[2], y[3]));
          }
        }
        // O^T += V^T P^T; lane's tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t v[4][VB / 4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const unsigned char* at = st + b * C::kBlockBytes + 16 * D +
                                      value_at<D>(2 * j + (e & 1) + 8 * (e >> 1), i8 * VB / 16) +
                                      (i8 * VB) % 16;
            if (VB == 16) {
              const uint4 y = *reinterpret_cast<const uint4*>(at);
              v[e][0] = y.x; v[e][1] = y.y; v[e][VB / 4 - 2] = y.z; v[e][VB / 4 - 1] = y.w;
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(at);
              v[e][0] = y.x; v[e][1] = y.y;
            }
            // what lies past the request's end may be a NaN
            if (CODE == KDA_E4M3 && EDGE && tok + 16 * b + 2 * j + (e & 1) + 8 * (e >> 1) >= kv) {
#pragma unroll
              for (int w = 0; w < VB / 4; ++w) v[e][w] = 0;
            }
          }
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            // channels 2 s and 2 s + 1 of two tokens
            const uint32_t sel = (s & 1) ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            codes_to_half<CODE>(__byte_perm(v[0][s >> 1], v[1][s >> 1], sel), a0, a1);
            codes_to_half<CODE>(__byte_perm(v[2][s >> 1], v[3][s >> 1], sel), a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(o[nt][s], a0, a1, a2, a3, pb[b][nt][0], pb[b][nt][1]);
          }
        }
      };
      if (edge)
        take(std::true_type{});
      else
        take(std::false_type{});
    }
    copy_wait<0>();
    __syncwarp();

    // the warps' sums meet in shared memory (each in its own ring)
    float* so = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float ov = pow2_inverse(vinv[nt][c]) * (1.0f / code_top(CODE));
        float y = l[nt][c];
        y += __shfl_xor_sync(~0u, y, 4);
        y += __shfl_xor_sync(~0u, y, 8);
        y += __shfl_xor_sync(~0u, y, 16);
        const int row = 8 * nt + 2 * j + c;
        if (i8 == 0) {
          s_m[warp][row] = y == 0.0f ? -INFINITY : m[nt][c];
          s_l[warp][row] = y;
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
          *reinterpret_cast<float2*>(so + row * D + i8 * VB + 2 * s) =
              make_float2(o[nt][s][c] * ov, o[nt][s][c + 2] * ov);
      }
    }
    __syncthreads();
    const bool last = b1 == mine1, whole = mine0 == 0 && mine1 == nb;
    const int64_t part = 2 * (int64_t)blockIdx.x + (mine0 > 0 ? 0 : 1);
    const int piece = (b0 - mine0) / C::kFold & 1;
    for (int e = tid; e < rows * D; e += kThreads) {
      const int row = e / D, ch = e % D;
      float* po = p.parts.o + (part * kFewRows + row) * D + ch;
      float mx = s_m[0][row];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][row]);
      if (b0 > mine0) mx = fmaxf(mx, s_sum[piece][row].x);
      const float mm = mx == -INFINITY ? 0.0f : mx;
      float sum = 0.0f, acc = 0.0f;
      if (b0 > mine0) {
        const float f = ex2(s_sum[piece][row].x - mm);
        sum = f * s_sum[piece][row].y;
        acc = f * *po;
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_m[w][row] - mm);
        sum += f * s_l[w][row];
        acc += f * *reinterpret_cast<float*>(smem + w * C::kWarpBytes + e * 4);
      }
      if (last && whole) {
        const int64_t at =
            (int64_t)(rq.c0 + (row0 + row) / G) * p.Hq + h * G + (row0 + row) % G;
        reinterpret_cast<__nv_bfloat16*>(p.out)[at * D + ch] =
            __float2bfloat16_rn(sum == 0.0f ? 0.0f : acc / sum);
        if (p.lse && ch == 0)
          p.lse[at] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
      } else {
        *po = acc;
        if (ch == 0) {
          s_sum[piece ^ 1][row] = make_float2(mx, sum);
          p.parts.ml[(part * kFewRows + row) * 2] = mx;
          p.parts.ml[(part * kFewRows + row) * 2 + 1] = sum;
        }
      }
    }
    __syncthreads();
    u = seg0 + b1;
  }
}

// Joins the parts of the segments that cross a worker's share, in the workers'
// order: out = sum_c w_c O_c / sum_c w_c l_c with w_c = 2^(m_c - max m).  Every
// block lists the segments for itself, by the boundaries between workers c and
// c + 1 that are the first inside theirs (one load a thread), and the blocks
// share out pieces of `group` rows, the fewest with which a block has one piece,
// 32 at most: a long cache leaves few rows with up to a part for each worker, a
// batch of prompts many rows with two or three.  Where the rows are at most half
// as many as a block's warps, several warps share a row's parts.  Bound by the
// parts' trip through L2 and by latency: with pieces of a fixed size, a block
// for each of every boundary's, one request with 100 000 tokens took 48 us (26
// so), a prompt's 128 tokens on 4000 41 (29), one with 700 tokens 11 (12).
constexpr int kJoinWarps = 16;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps, 2)
    kda_attn_join_kernel(AttnArgs p, Parts rows_kernel, Parts tile_kernel) {
  constexpr int E = D / 32, NT = 32 * kJoinWarps;
  __shared__ float s_o[kJoinWarps][D], s_l[kJoinWarps];
  // first and last worker, first token, rows, first row and head of the segments
  __shared__ int4 s_few[kRowsPerSm * kMaxSms], s_tile[kMaxSms / 2];
  __shared__ int s_count[kJoinWarps], s_rows[kJoinWarps], s_most[kJoinWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_kernel_before();
  int count[2], most[2] = {1, 1}, rows_all = 0;  // (most: rows of one segment)
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Parts& q = k ? tile_kernel : rows_kernel;
    count[k] = 0;
    if (q.ctas < 2) continue;
    const int64_t total = *q.total;
    for (int base = 0; base < q.ctas - 1; base += NT) {
      const int c = base + tid;
      PartHead h{0, 0, 0, 0, 0, 0};
      if (c < q.ctas - 1) h = q.head[c + 1];
      const int64_t share = quotient(total + q.ctas - 1, q.ctas);
      const int rows = h.rows > 0 && quotient(h.seg0, share) == c ? h.rows : 0;
      const uint32_t those = __ballot_sync(~0u, rows > 0);
      const int sum = __reduce_add_sync(~0u, rows), top = __reduce_max_sync(~0u, rows);
      if (lane == 0) {
        s_count[warp] = __popc(those);
        s_rows[warp] = sum;
        s_most[warp] = top;
      }
      __syncthreads();
      int at = count[k] + __popc(those & ((1u << lane) - 1));
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        if (w < warp) at += s_count[w];
        count[k] += s_count[w];
        rows_all += s_rows[w];
        most[k] = max(most[k], s_most[w]);
      }
      if (rows > 0)
        (k ? s_tile : s_few)[at] = make_int4(c | (int)quotient(h.seg1 - 1, share) << 16, h.tok0,
                                             rows | h.row0 << 16, h.h);
      __syncthreads();
    }
  }
  int group = 1;
  while (group < 32 && rows_all > group * (int)gridDim.x) group *= 2;
  const int few_groups = (most[0] + group - 1) / group, tile_groups = (most[1] + group - 1) / group;
  const int few_items = count[0] * few_groups, items = few_items + count[1] * tile_groups;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const bool few = item < few_items;
    const Parts& q = few ? rows_kernel : tile_kernel;
    const int of = few ? item : item - few_items, groups = few ? few_groups : tile_groups;
    const int4 seg = (few ? s_few : s_tile)[of / groups];
    const int ca = seg.x & 0xffff, cb = seg.x >> 16, row0 = group * (of % groups);
    const int n = min((seg.z & 0xffff) - row0, group);
    if (n <= 0) continue;
    int wpr = 1;  // warps a row
    while (2 * n * wpr <= kJoinWarps) wpr *= 2;
    const int sub = warp % wpr;
    for (int i = warp / wpr; i < n; i += kJoinWarps / wpr) {
      const int row = row0 + i;
      // the first CTA holds it as its last segment, the others as their first
      auto part = [&](int c) -> int64_t {
        return (2 * (int64_t)c + (c == ca ? 1 : 0)) * q.rows + row;
      };
      float mx = -INFINITY, acc[E] = {}, sum = 0.0f;
      for (int c = ca + lane; c <= cb; c += 32) mx = fmaxf(mx, q.ml[part(c) * 2]);
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
      const float mm = mx == -INFINITY ? 0.0f : mx;
#pragma unroll 8
      for (int c = ca + sub; c <= cb; c += wpr) {
        const int64_t at = part(c);
        const float2 ml = *reinterpret_cast<const float2*>(q.ml + at * 2);
        const float f = ex2(ml.x - mm);
        sum += f * ml.y;
        float v[E];
        if constexpr (E == 4)
          *reinterpret_cast<float4*>(v) = reinterpret_cast<const float4*>(q.o + at * D)[lane];
        else
          *reinterpret_cast<float2*>(v) = reinterpret_cast<const float2*>(q.o + at * D)[lane];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += f * v[e];
      }
      if (wpr > 1) {  // (then each warp has one row at most)
#pragma unroll
        for (int e = 0; e < E; ++e) s_o[warp][E * lane + e] = acc[e];
        if (lane == 0) s_l[warp] = sum;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / wpr), "r"(32 * wpr) : "memory");
        if (sub) break;
        for (int w = 1; w < wpr; ++w) {
          sum += s_l[warp + w];
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] += s_o[warp + w][E * lane + e];
        }
      }
      const int of_seg = (seg.z >> 16) + row;
      const int64_t at = (int64_t)(seg.y + of_seg / p.G) * p.Hq + seg.w * p.G + of_seg % p.G;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      uint32_t y[E / 2];
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const __nv_bfloat162 z = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
        y[e / 2] = *reinterpret_cast<const uint32_t*>(&z);
      }
      if constexpr (E == 4)
        reinterpret_cast<uint2*>(p.out + at * D)[lane] = make_uint2(y[0], y[1]);
      else
        reinterpret_cast<uint32_t*>(p.out + at * D)[lane] = y[0];
      if (p.lse && lane == 0)
        p.lse[at] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
    }
    __syncthreads();
  }
}

template <int CODE, int D, int NT>
kda_status launch_rows(const AttnArgs& p, cudaStream_t s) {
  auto kernel = kda_cache_attn_rows_kernel<CODE, D, NT>;
  const int smem = kWarps * Cfg<D, NT>::kWarpBytes;
  const kda_status rc = kda_smem_attr((const void*)kernel, smem);
  if (rc != KDA_OK) return rc;
  kernel<<<p.parts.ctas, kThreads, smem, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <int CODE, int D>
kda_status launch_nt(const AttnArgs& p, cudaStream_t s) {
  // one 8-row tile where no request can have more rows than that: two, the
  // second empty, take 148 us where one takes 139 (64 decode steps of 4 rows, int8;
  // e4m3 142 and 137)
  if ((int64_t)p.max_new * p.G <= 8) return launch_rows<CODE, D, 1>(p, s);
  return launch_rows<CODE, D, 2>(p, s);
}

}  // namespace

kda_status kda_launch_attn_rows(const AttnArgs& p, int d, int code, cudaStream_t s) {
  if (code == KDA_I8) return d == 64 ? launch_nt<KDA_I8, 64>(p, s) : launch_nt<KDA_I8, 128>(p, s);
  return d == 64 ? launch_nt<KDA_E4M3, 64>(p, s) : launch_nt<KDA_E4M3, 128>(p, s);
}

kda_status kda_launch_attn_join(const AttnArgs& p, const Parts& tile, int d, cudaStream_t s) {
  // two blocks an SM, or one for each row of the batch where these are fewer
  const int64_t rows = (int64_t)p.T * p.Hq, most = 2 * (p.parts.ctas / kRowsPerSm);
  const int blocks = (int)(rows < most ? rows : most);
  return launch_following(d == 64 ? kda_attn_join_kernel<64> : kda_attn_join_kernel<128>, blocks,
                          32 * kJoinWarps, 0, s, p, p.parts, tile);
}
