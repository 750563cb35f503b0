// kda_cache.cu -- the paged 8-bit cache's bookkeeping and its write side:
// the page plan of a step, the release of finished requests, the append of
// a step's keys and values.
#include "kda_cache.cuh"

namespace {

using namespace kda_cache;

// ---------------------------------------------------------------------------
// block-wide inclusive scan of three 64-bit sums, NT threads

struct Sums {
  int64_t tok, page, run;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.tok + b.tok, a.page + b.page, a.run + b.run};
}

// Exclusive prefix of each thread's x; `total` gets the sum of all.
template <int NT>
__device__ Sums block_scan(Sums x, Sums* s_warp, Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Sums y{__shfl_up_sync(~0u, inc.tok, o), __shfl_up_sync(~0u, inc.page, o),
           __shfl_up_sync(~0u, inc.run, o)};
    if (lane >= o) inc = inc + y;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  Sums before{0, 0, 0};
  total = {0, 0, 0};
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before = before + s_warp[w];
    total = total + s_warp[w];
  }
  return {before.tok + inc.tok - x.tok, before.page + inc.page - x.page,
          before.run + inc.run - x.run};
}

// The last index i in [0, n) with a[i] <= x (a non-decreasing, a[0] <= x).
// Several i may share a value when requests bring nothing: the last of them
// is the one whose range holds x.
__device__ __forceinline__ int last_not_above(const int32_t* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// page plan

struct PlanArgs {
  const int32_t *new_lens, *ctx_lens, *free_pages, *free_count;
  int32_t *table, *cu, *kv_lens, *slots, *positions, *runs, *free_out, *status;
  int R, T, page_log2, max_pages, num_pages, max_runs;
};

constexpr int kPlanThreads = 512;

// Three prefix sums over the requests (new tokens, pages taken, runs), then
// every token, page and run finds its request by binary search.  Every CTA
// scans the lengths itself (R integers that stay in L2), so the whole plan
// is one launch and no CTA waits for another; CTA 0 writes what is per
// request.  Nothing that another CTA reads is written: fresh table columns
// are computed from the stack by whoever needs them, not read back.
// Bound by latency (a chain of dependent loads and two barriers): 4.1 us for 64
// requests' decode step, 4.7 us for 17 prompts with 37 000 tokens.
__global__ void __launch_bounds__(kPlanThreads) kda_page_plan_kernel(PlanArgs p) {
  extern __shared__ int32_t sm[];
  int32_t* s_tok = sm;                 // [R] first packed row
  int32_t* s_page = sm + p.R;          // [R] pages taken by the requests before
  int32_t* s_run = sm + 2 * p.R;       // [R] runs of the requests before
  __shared__ Sums s_warp[kPlanThreads / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, R = p.R, lg = p.page_log2, P = 1 << lg;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const int per = (R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  const int64_t cap = (int64_t)p.max_pages << lg;
  auto of = [&](int r, bool& ok) -> Sums {
    const int64_t n = p.new_lens[r], c = p.ctx_lens[r];
    ok = n >= 0 && c >= 0 && n + c <= cap && n <= p.T;
    if (!ok) return {0, 0, 0};
    const int64_t before = (c + P - 1) >> lg, after = (n + c + P - 1) >> lg;
    return {n, after - before, n > 0 ? after - (c >> lg) : 0};
  };
  Sums mine{0, 0, 0}, total;
  for (int r = r0; r < r1; ++r) {
    bool ok;
    mine = mine + of(r, ok);
    if (!ok) s_bad = 1;
  }
  Sums at = block_scan<kPlanThreads>(mine, s_warp, total);
  const int left = p.free_count[0];
  const bool bad_lens = s_bad != 0 || total.tok > p.T;  // (after block_scan's barrier)
  const bool no_pages = left < 0 || left > p.num_pages || total.page > left;
  const bool ok = !bad_lens && !no_pages;
  for (int r = r0; r < r1; ++r) {
    bool fine;
    s_tok[r] = (int32_t)at.tok;
    s_page[r] = (int32_t)at.page;
    s_run[r] = (int32_t)at.run;
    at = at + of(r, fine);
  }
  __syncthreads();
  const int n_tok = ok ? (int)total.tok : 0, n_page = ok ? (int)total.page : 0;
  const int n_run = ok ? (int)total.run : 0;
  const int gtid = blockIdx.x * kPlanThreads + tid, gsize = gridDim.x * kPlanThreads;

  // the page in column c of request r, whether held before or taken now
  auto page_of = [&](int r, int ctx, int c) {
    const int before = (ctx + P - 1) >> lg;
    if (c < before) return p.table[(int64_t)r * p.max_pages + c];
    return p.free_pages[left - 1 - (s_page[r] + c - before)];
  };
  for (int t = gtid; t < p.T; t += gsize) {
    int slot = -1, pos = -1;
    if (t < n_tok) {
      const int r = last_not_above(s_tok, R, t), ctx = p.ctx_lens[r];
      pos = ctx + t - s_tok[r];
      const int pg = page_of(r, ctx, pos >> lg);
      if (pg >= 0 && pg < p.num_pages) slot = (pg << lg) + (pos & (P - 1));
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
  for (int i = gtid; i < n_page; i += gsize) {
    const int r = last_not_above(s_page, R, i), ctx = p.ctx_lens[r];
    const int col = ((ctx + P - 1) >> lg) + i - s_page[r];
    p.table[(int64_t)r * p.max_pages + col] = p.free_pages[left - 1 - i];
  }
  for (int j = gtid; j < p.max_runs; j += gsize) {
    int4 run = make_int4(0, 0, 0, 0);
    if (j < n_run) {
      const int r = last_not_above(s_run, R, j), ctx = p.ctx_lens[r];
      const int kv = ctx + p.new_lens[r], col = (ctx >> lg) + j - s_run[r];
      const int a = max(col << lg, ctx), b = min((col << lg) + P, kv);
      const int pg = page_of(r, ctx, col);
      if (pg >= 0 && pg < p.num_pages)
        run = make_int4(s_tok[r] + a - ctx, b - a, pg, a & (P - 1));
      else
        report(p.status, KDA_ERR_BAD_PAGES);
    }
    reinterpret_cast<int4*>(p.runs)[j] = run;
  }
  if (blockIdx.x == 0) {
    for (int r = tid; r < R; r += kPlanThreads) {
      p.cu[r] = ok ? s_tok[r] : 0;
      p.kv_lens[r] = p.ctx_lens[r] + (ok ? p.new_lens[r] : 0);
    }
    if (tid == 0) {
      p.cu[R] = n_tok;
      p.free_out[0] = left - n_page;
      if (!ok) report(p.status, bad_lens ? KDA_ERR_BAD_SEQLENS : KDA_ERR_NO_PAGES);
    }
  }
}

// ---------------------------------------------------------------------------
// release

struct ReleaseArgs {
  const int32_t* release;
  int32_t *kv_lens, *table, *free_pages, *free_count, *status;
  int R, page_log2, max_pages, num_pages;
};

// One CTA: the pages of finished requests are few, and one CTA needs no
// order among others to update the stack in place.  Bound by latency: 2.1 us for
// one of 64 requests with 128 pages each, 15 us for all of them (1.7 and 10 without
// the look at all pages before any is moved).
__global__ void __launch_bounds__(kPlanThreads) kda_page_release_kernel(ReleaseArgs p) {
  extern __shared__ int32_t s_first[];  // [R] pages pushed by the requests before
  __shared__ Sums s_warp[kPlanThreads / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, R = p.R, P = 1 << p.page_log2;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const int per = (R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  auto pages = [&](int r) -> int64_t {
    if (!p.release[r]) return 0;
    return ((int64_t)p.kv_lens[r] + P - 1) >> p.page_log2;
  };
  Sums mine{0, 0, 0}, total;
  for (int r = r0; r < r1; ++r) {
    const int64_t n = pages(r);
    if (n < 0 || n > p.max_pages || p.kv_lens[r] < 0) s_bad = 1;
    mine.page += n;
  }
  Sums at = block_scan<kPlanThreads>(mine, s_warp, total);
  const int64_t held = p.free_count[0];
  const bool bad_lens = s_bad != 0;
  const bool full = held < 0 || held + total.page > p.num_pages;
  if (bad_lens || full) {
    if (tid == 0) report(p.status, bad_lens ? KDA_ERR_BAD_SEQLENS : KDA_ERR_BAD_PAGES);
    return;
  }
  for (int r = r0; r < r1; ++r) {
    s_first[r] = (int32_t)at.page;
    at.page += pages(r);
  }
  __syncthreads();
  auto entry = [&](int i) {
    const int r = last_not_above(s_first, R, i);
    return p.table + (int64_t)r * p.max_pages + (i - s_first[r]);
  };
  bool in = true;  // (a page outside the pool would be handed out again)
  for (int i = tid; i < (int)total.page; i += kPlanThreads)
    in &= (uint32_t)*entry(i) < (uint32_t)p.num_pages;
  if (!__syncthreads_and(in)) {
    if (tid == 0) report(p.status, KDA_ERR_BAD_PAGES);
    return;
  }
  for (int i = tid; i < (int)total.page; i += kPlanThreads) {
    int32_t* e = entry(i);
    p.free_pages[held + i] = *e;
    *e = -1;
  }
  __syncthreads();
  for (int r = tid; r < R; r += kPlanThreads)
    if (p.release[r]) p.kv_lens[r] = 0;
  if (tid == 0) p.free_count[0] = (int32_t)(held + total.page);
}

// ---------------------------------------------------------------------------
// append

struct AppendArgs {
  const uint16_t* x[2];  // k, v
  int64_t stride[2];
  uint8_t* codes[2];
  float* scale[2];
  const int32_t* runs;
  int32_t* status;
  int T, num_pages, H;
};

// Threads: kAppendPasses 16-byte pieces each where the page has so many.  More
// pieces a thread are more bytes in flight an SM until registers run out: the
// prompts' append took 48.0 / 41.0 / 44.5 us with 4 / 8 / 16 (e4m3; int8 41.3 with 8).
constexpr int kAppendPasses = 8;
__host__ __device__ constexpr int append_threads(int page, int d) {
  const int n = page * d / 8 / kAppendPasses;
  return n < 64 ? 64 : n > 512 ? 512 : n;
}

// Codes of 8 bf16 values (as 4 words): rn(x TOP / a), exactly and without a
// division; inv = TOP / (a pre).  t = (x pre) inv is within 2^-23 of the
// quotient (two roundings), which so lies between t (1 - 2^-22) and
// t (1 + 2^-22); rounding to a code is monotonic, and where both ends give the
// same code that is the one.  Where they differ the quotient is a tie, and the
// even code is taken: x and a have 8 significant bits, so a quotient that is
// no tie keeps a relative distance of 2^-16 (int8: |127 X 2^k - (2 n + 1) A| is
// a whole multiple of the smaller unit, against at most 2 A 127) or 2^-13
// (e4m3: the same with 7 X and M A, M at most 31) from every tie.
template <int CODE>
__device__ __forceinline__ uint2 encode8(const uint32_t (&w)[4], float pre, float inv) {
  float lo[8], hi[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float f = __uint_as_float((e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    const float t = f * pre * inv;
    lo[e] = t * (1.0f - 0x1p-22f);
    hi[e] = t * (1.0f + 0x1p-22f);
  }
  uint32_t a[2], b[2];
  if (CODE == KDA_I8) {
    // (adding 1.5 * 2^23 rounds to an integer, ties to even, in the low bits)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = __float_as_uint(lo[4 * i + e] + 12582912.0f);
        y[e] = __float_as_uint(hi[4 * i + e] + 12582912.0f);
      }
      a[i] = __byte_perm(__byte_perm(x[0], x[1], 0x0040), __byte_perm(x[2], x[3], 0x0040), 0x5410);
      b[i] = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t x[2], y[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int at = 4 * i + 2 * e;
        x[e] = __nv_cvt_float2_to_fp8x2(make_float2(lo[at], lo[at + 1]), __NV_SATFINITE, __NV_E4M3);
        y[e] = __nv_cvt_float2_to_fp8x2(make_float2(hi[at], hi[at + 1]), __NV_SATFINITE, __NV_E4M3);
      }
      a[i] = x[0] | x[1] << 16;
      b[i] = y[0] | y[1] << 16;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t odd = (a[i] & 0x01010101u) * 0xffu;
    a[i] ^= (a[i] ^ b[i]) & odd;
  }
  return make_uint2(a[0], a[1]);
}

// One CTA per (run, head, tensor).  The run's values are read once, into
// registers, their largest magnitude is found by an unsigned maximum of the bit
// patterns without the sign (which orders finite < infinity < NaN), and the
// codes are written from the registers.  A stream of 3 bytes a value: 17 prompts
// with 37 000 tokens of 8 heads (230 MB) take 41.0 us, 5.6 TB/s; one token of
// each of 64 requests 3.5 us, which is latency.
template <int CODE, int D, int PAGE>
__global__ void __launch_bounds__(append_threads(PAGE, D))
    kda_cache_append_kernel(AppendArgs p) {
  constexpr int NT = append_threads(PAGE, D);
  constexpr int TPR = D / 8;     // threads per token, 8 values each
  constexpr int RPP = NT / TPR;  // tokens per pass
  constexpr int PASSES = PAGE / RPP;
  constexpr float TOP = code_top(CODE);
  __shared__ uint32_t s_max[NT / 32];
  const int tid = threadIdx.x;
  const int which = blockIdx.x % (2 * p.H), j = blockIdx.x / (2 * p.H);
  const int h = which >> 1, kv = which & 1;
  const int4 run = reinterpret_cast<const int4*>(p.runs)[j];
  const int row = run.x, count = run.y, page = run.z, off = run.w;
  if (count == 0) return;
  if (count < 0 || count > PAGE || off < 0 || off + count > PAGE || page < 0 ||
      page >= p.num_pages || row < 0 || row > p.T - count) {
    if (tid == 0) report(p.status, KDA_ERR_BAD_PAGES);
    return;
  }
  // (an index into the arguments would copy them to local memory)
  const int64_t stride = kv ? p.stride[1] : p.stride[0];
  const uint16_t* x = (kv ? p.x[1] : p.x[0]) + (int64_t)row * stride + h * D + (tid % TPR) * 8;
  uint8_t* codes =
      (kv ? p.codes[1] : p.codes[0]) + ((int64_t)page * p.H + h) * (PAGE * D) + (tid % TPR) * 8;
  float* scale = (kv ? p.scale[1] : p.scale[0]) + (int64_t)page * p.H + h;
  const int t0 = tid / TPR;

  uint4 v[PASSES];
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    const int t = t0 + i * RPP;
    if (t < count) v[i] = *reinterpret_cast<const uint4*>(x + t * stride);
  }
  const uint32_t had = off > 0 ? __float_as_uint(*scale) & 0x7fffffffu : 0;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      most = max(most, max(w[e] & 0x7fff0000u, (w[e] << 16) & 0x7fff0000u));
  }
  most = __reduce_max_sync(~0u, most);
  if ((tid & 31) == 0) s_max[tid >> 5] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) most = max(most, s_max[w]);
  const uint32_t now = max(most, had);
  const bool poisoned = now >= 0x7f800000u;
  if (tid == 0) *scale = poisoned ? __uint_as_float(0x7fc00000u) : __uint_as_float(now);
  const float a1 = __uint_as_float(now), a0 = __uint_as_float(had);
  // a power of two on both sides of a quotient keeps its terms finite and
  // normal; it changes no quotient
  const float pre = now >= 0x5f800000u ? 0x1p-64f : now < 0x1f800000u ? 0x1p64f : 1.0f;
  const float den = a1 * pre;
  const float inv = TOP / den;
  if (now != had && had != 0 && !poisoned) {
    for (int t = t0; t < off; t += RPP) {
      uint2 c = *reinterpret_cast<uint2*>(codes + t * D);
      uint32_t w[2] = {c.x, c.y}, r[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q = decode1<CODE>((uint8_t)(w[e >> 2] >> (8 * (e & 3))));
        r[e >> 2] |= encode1<CODE>(__fdiv_rn(q * (a0 * pre), den)) << (8 * (e & 3));
      }
      *reinterpret_cast<uint2*>(codes + t * D) = make_uint2(r[0], r[1]);
    }
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int t = t0 + i * RPP;
    if (t >= count) break;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint2 r = make_uint2(0, 0);
    if (now != 0 && !poisoned) r = encode8<CODE>(w, pre, inv);
    *reinterpret_cast<uint2*>(codes + (int64_t)(off + t) * D) = r;
  }
}

template <int CODE, int D>
void launch_append(const AppendArgs& p, int page, unsigned grid, cudaStream_t s) {
  switch (page) {
    case 16: kda_cache_append_kernel<CODE, D, 16><<<grid, append_threads(16, D), 0, s>>>(p); break;
    case 32: kda_cache_append_kernel<CODE, D, 32><<<grid, append_threads(32, D), 0, s>>>(p); break;
    case 64: kda_cache_append_kernel<CODE, D, 64><<<grid, append_threads(64, D), 0, s>>>(p); break;
    default: kda_cache_append_kernel<CODE, D, 128><<<grid, append_threads(128, D), 0, s>>>(p);
  }
}

int log2_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

kda_status clear_status(int32_t* dev_status, cudaStream_t s) {
  if (!dev_status) return KDA_OK;
  return cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) == cudaSuccess ? KDA_OK
                                                                           : KDA_ERR_CUDA;
}

}  // namespace

extern "C" int kda_page_runs(int R, int T, int page) {
  if (R < 1 || T < 0 || !page_ok(page)) return 0;
  const int64_t n = (int64_t)T / page + 2 * (int64_t)R;
  return (int)(n < T ? n : T > 0 ? T : 1);
}

extern "C" kda_status kda_page_plan(const int32_t* new_lens, const int32_t* ctx_lens, int R,
                                    int T, int page, int32_t* block_table, int max_pages,
                                    const int32_t* free_pages, const int32_t* free_count,
                                    int num_pages, int32_t* cu_seqlens, int32_t* kv_lens,
                                    int32_t* slots, int32_t* positions, int32_t* runs,
                                    int32_t* free_count_out, int32_t* dev_status,
                                    kda_stream_t stream) {
  if (!new_lens || !ctx_lens || !block_table || !free_pages || !free_count || !cu_seqlens ||
      !kv_lens || !runs || !free_count_out || R < 1 || T < 0 || max_pages < 1 || num_pages < 1)
    return KDA_ERR_INVALID_ARG;
  if (T > 0 && (!slots || !positions)) return KDA_ERR_INVALID_ARG;
  if (R > kMaxRequests || !page_ok(page)) return KDA_ERR_UNSUPPORTED;
  if ((int64_t)num_pages * page > INT32_MAX || (int64_t)max_pages * page > (1 << 30) ||
      T > (1 << 26))
    return KDA_ERR_UNSUPPORTED;  // slots and lengths are int32
  if (!aligned(16, runs) || !aligned(4, new_lens, ctx_lens, block_table, free_pages, free_count,
                                     cu_seqlens, kv_lens, slots, positions, free_count_out,
                                     dev_status))
    return KDA_ERR_MISALIGNED;
  const int max_runs = kda_page_runs(R, T, page);
  const size_t n4 = sizeof(int32_t);
  const void* outs[] = {cu_seqlens, kv_lens, slots, positions, runs, free_count_out};
  const size_t out_n[] = {(R + 1) * n4, R * n4, T * n4, T * n4, max_runs * 4 * n4, n4};
  const void* ins[] = {new_lens, ctx_lens, free_pages, free_count, block_table};
  const size_t in_n[] = {R * n4, R * n4, num_pages * n4, n4, (size_t)R * max_pages * n4};
  for (int o = 0; o < 6; ++o)
    for (int i = 0; i < 5; ++i)
      if (overlaps(outs[o], out_n[o], ins[i], in_n[i])) return KDA_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (overlaps(ins[i], in_n[i], block_table, in_n[4])) return KDA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int smem = 3 * R * (int)n4;
  if (smem > 40 * 1024) {
    kda_status rc = kda_smem_attr((const void*)kda_page_plan_kernel, smem);
    if (rc != KDA_OK) return rc;
  }
  const int sms = kda_device_sms();
  if (sms < 1) return KDA_ERR_CUDA;
  kda_status rc = clear_status(dev_status, s);
  if (rc != KDA_OK) return rc;
  PlanArgs p{new_lens, ctx_lens, free_pages, free_count, block_table, cu_seqlens, kv_lens, slots,
             positions, runs, free_count_out, dev_status, R, T, log2_of(page), max_pages,
             num_pages, max_runs};
  const int work = T > R ? T : R;
  int grid = (work + 2 * kPlanThreads - 1) / (2 * kPlanThreads);
  grid = grid < 1 ? 1 : grid > sms ? sms : grid;
  kda_page_plan_kernel<<<grid, kPlanThreads, smem, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status kda_page_release(const int32_t* release, int R, int page, int32_t* kv_lens,
                                       int32_t* block_table, int max_pages, int32_t* free_pages,
                                       int32_t* free_count, int num_pages, int32_t* dev_status,
                                       kda_stream_t stream) {
  if (!release || !kv_lens || !block_table || !free_pages || !free_count || R < 1 ||
      max_pages < 1 || num_pages < 1)
    return KDA_ERR_INVALID_ARG;
  if (R > kMaxRequests || !page_ok(page)) return KDA_ERR_UNSUPPORTED;
  if (!aligned(4, release, kv_lens, block_table, free_pages, free_count, dev_status))
    return KDA_ERR_MISALIGNED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int smem = R * (int)sizeof(int32_t);
  if (smem > 40 * 1024) {
    kda_status rc = kda_smem_attr((const void*)kda_page_release_kernel, smem);
    if (rc != KDA_OK) return rc;
  }
  kda_status rc = clear_status(dev_status, s);
  if (rc != KDA_OK) return rc;
  ReleaseArgs p{release, kv_lens, block_table, free_pages, free_count, dev_status, R,
                log2_of(page), max_pages, num_pages};
  kda_page_release_kernel<<<1, kPlanThreads, smem, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status kda_cache_append(const uint16_t* k, const uint16_t* v, int64_t k_stride,
                                       int64_t v_stride, int T, const int32_t* runs, int num_runs,
                                       void* k_codes, void* v_codes, float* k_scale,
                                       float* v_scale, int num_pages, int page, int Hkv, int d,
                                       kda_code code, int32_t* dev_status, kda_stream_t stream) {
  if (T < 0 || num_runs < 0 || num_pages < 1 || Hkv < 1) return KDA_ERR_INVALID_ARG;
  if (!runs || !k_codes || !v_codes || !k_scale || !v_scale) return KDA_ERR_INVALID_ARG;
  if (T > 0 && (!k || !v)) return KDA_ERR_INVALID_ARG;
  if (!page_ok(page) || !head_dim_ok(d) || (code != KDA_I8 && code != KDA_E4M3) || Hkv > 4096 ||
      T > (1 << 26))
    return KDA_ERR_UNSUPPORTED;
  const int64_t width = (int64_t)Hkv * d;
  if (k_stride < width || v_stride < width) return KDA_ERR_INVALID_ARG;
  if (k_stride % 8 || v_stride % 8 || !aligned(16, k, v, k_codes, v_codes, runs) ||
      !aligned(4, k_scale, v_scale, dev_status))
    return KDA_ERR_MISALIGNED;
  const size_t pool = (size_t)num_pages * width * page, sc = (size_t)num_pages * Hkv * 4;
  const void* outs[] = {k_codes, v_codes, k_scale, v_scale};
  const size_t out_n[] = {pool, pool, sc, sc};
  const void* ins[] = {k, v, runs};
  const size_t in_n[] = {T ? (size_t)((T - 1) * k_stride + width) * 2 : 0,
                         T ? (size_t)((T - 1) * v_stride + width) * 2 : 0, (size_t)num_runs * 16};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 3; ++i)
      if (overlaps(outs[o], out_n[o], ins[i], in_n[i])) return KDA_ERR_INVALID_ARG;
    for (int i = o + 1; i < 4; ++i)
      if (overlaps(outs[o], out_n[o], outs[i], out_n[i])) return KDA_ERR_INVALID_ARG;
  }
  const int64_t grid = (int64_t)num_runs * 2 * Hkv;
  if (grid > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  kda_status rc = clear_status(dev_status, s);
  if (rc != KDA_OK) return rc;
  // (without rows every run is outside them)
  if (grid == 0 || (T == 0 && !dev_status)) return KDA_OK;
  AppendArgs p{{k, v}, {k_stride, v_stride}, {(uint8_t*)k_codes, (uint8_t*)v_codes},
               {k_scale, v_scale}, runs, dev_status, T, num_pages, Hkv};
  const unsigned g = (unsigned)grid;
  if (code == KDA_I8) {
    if (d == 64) launch_append<KDA_I8, 64>(p, page, g, s);
    else launch_append<KDA_I8, 128>(p, page, g, s);
  } else {
    if (d == 64) launch_append<KDA_E4M3, 64>(p, page, g, s);
    else launch_append<KDA_E4M3, 128>(p, page, g, s);
  }
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
