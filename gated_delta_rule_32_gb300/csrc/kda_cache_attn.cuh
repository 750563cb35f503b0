// kda_cache_attn.cuh -- what the attention kernels over the paged cache
// share: arguments, the requests' checks, the schedule and the partial
// results.
#pragma once

#include "kda_cache.cuh"

namespace kda_cache {

// The segment (request, head, row tile) that a CTA's share begins in the
// middle of: its units, first token, rows (0: none) and head.
struct PartHead {
  int64_t seg0, seg1;
  int32_t tok0, rows, h, row0;  // (row0: its first row, counted from tok0)
};

// What a kernel leaves for the join, in the workspace.  A worker leaves at most
// two parts: of the segment that its share begins in (slot 2 c) and of the one
// that it ends in (slot 2 c + 1).  A long run of tokens is put together in the same
// slot, piece by piece; the tile kernel's pieces come through a third one (2 ctas + c).
struct Parts {
  int ctas, rows;    // workers of the kernel (CTAs, or pairs); a part's rows
  int64_t* total;    // units of the whole batch
  PartHead* head;    // [ctas]
  float* ml;         // [slot][rows][2] maximum (log2) and sum of a part's rows
  float* o;          // [slot][rows][D] a part's sum of weighted values
};

struct AttnArgs {
  const uint16_t* q;
  int64_t q_stride;
  const int32_t *cu, *kv_lens, *table;
  const uint8_t *k_codes, *v_codes;
  const float *k_scale, *v_scale;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int R, T, max_new, max_pages, Hq, Hkv, G, num_pages, page_log2, few_max;
  float scale;
  Parts parts;  // of the kernel that the arguments are for
};

// A request with at most few_max(d) query rows per key / value head runs on the
// few-row kernel, in groups of kFewRows.  Every group converts all codes once
// more, so its time grows with rows times d, the tile kernel's hardly up to its
// 512-row segments.  Few-row against tile kernel, us (e4m3): d = 64, 2 heads: 32
// requests with up to 4096 cached tokens, 64 rows 38 : 47, 96 rows 49 : 48, 128 rows
// 61 : 49; 4 requests with up to 65536, 64 rows 46 : 67, 128 rows 71 : 68.  d = 128: 48
// requests with up to 3000, 4 heads, 32 rows 73 : 98, 48 rows 97 : 96; 4 requests with up
// to 65536, 2 heads, 32 rows 52 : 79, 48 rows 64 : 79, 64 rows 74 : 80; single tokens of
// 64 requests with up to 8192, 48 rows 113 : 133.  (So the rule is right for short
// contexts, and 16 to 32 rows low for long ones.)
constexpr int kFewRows = 16;
__host__ __device__ constexpr int few_max(int d) { return 4096 / d; }
// CTAs of the few-row kernel an SM: as many as its registers allow.  SMs that the
// kernels use at most (what the join has room for).
constexpr int kRowsPerSm = 3, kMaxSms = 256;
// Query rows of a segment on the tile kernel.
constexpr int kTileRows = 512;

struct Req {
  int c0, n, kv;
};

// a / b of non-negative numbers, by the much shorter 32-bit division where it will do.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// Request r, or n = 0 if it brings nothing or is malformed (`bad`).
__device__ __forceinline__ Req load_req(const AttnArgs& p, int r, bool& bad) {
  const int a = p.cu[r], b = p.cu[r + 1], kv = p.kv_lens[r];
  bad = a < 0 || b < a || b > p.T || b - a > p.max_new || kv < 0 ||
        kv > ((int64_t)p.max_pages << p.page_log2);
  return {a, bad ? 0 : b - a, kv};
}

// The schedule: every request has a number of work units, the workers (CTAs, or
// pairs of them) take equal contiguous shares of the sum over requests.  A CTA
// finds the request its first unit falls in: every thread sums a contiguous
// range of requests, the block scans the sums, the thread whose range holds
// the unit walks it.  Worker 0 also writes the sum and reports malformed
// requests.  units(Req) -> int64; NT threads.  Returns the worker's units
// [u0, u1) and the request of u0 with the units before it; u0 == u1 if there
// is nothing to do.
struct Share {
  int64_t u0, u1, base;
  int r;
};

template <int NT, class Units>
__device__ __forceinline__ Share find_share(const AttnArgs& p, int worker, Units units) {
  __shared__ int64_t s_warp[NT / 32];
  __shared__ int64_t s_base;
  __shared__ int s_r;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.R + NT - 1) / NT;
  const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) {
    bool bad;
    const Req q = load_req(p, r, bad);
    if (bad && worker == 0) report(p.status, KDA_ERR_BAD_SEQLENS);
    if (q.n > 0) mine += units(q);
  }
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  const int64_t share = quotient(total + p.parts.ctas - 1, p.parts.ctas);
  Share s;
  s.u0 = min(total, (int64_t)worker * share);
  s.u1 = min(total, s.u0 + share);
  int64_t at = before + inc - mine;
  const bool here = s.u0 < s.u1 && at <= s.u0 && s.u0 < at + mine;
  if (here) {
    for (int r = r0; r < r1; ++r) {
      bool bad;
      const Req q = load_req(p, r, bad);
      const int64_t u = q.n > 0 ? units(q) : 0;
      if (at <= s.u0 && s.u0 < at + u) {
        s_r = r;
        s_base = at;
      }
      at += u;
    }
  }
  if (worker == 0 && tid == 0) *p.parts.total = total;
  __syncthreads();
  s.r = s_r;
  s.base = s_base;
  return s;
}

// Loads that are zero (or -1) where `use` is false: predicated, so that
// nothing waits for them before their value is used.
template <int OFFSET>
__device__ __forceinline__ uint4 load16_if(const void* src, bool use) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n"
      " mov.b32 %2, 0;\n mov.b32 %3, 0;\n @p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4 + %6];\n}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(src), "r"((int)use), "n"(OFFSET));
  return v;
}
__device__ __forceinline__ int load_page_if(const int32_t* src, bool use) {
  int v;
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n mov.b32 %0, -1;\n"
               " @p ld.global.nc.u32 %0, [%1];\n}"
               : "=&r"(v)
               : "l"(src), "r"((int)use));
  return v;
}
__device__ __forceinline__ float load_scale_if(const float* src, bool use) {
  float v;
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n mov.b32 %0, 0;\n"
               " @p ld.global.nc.f32 %0, [%1];\n}"
               : "=&f"(v)
               : "l"(src), "r"((int)use));
  return v;
}

// The smallest power of two not below x, from 2^-126 to 2^126 (of which x may so
// be up to four times as much), and the reciprocal of such a power (a division
// takes its slow path at the range's ends).
__device__ __forceinline__ float pow2_above(float x) {
  const uint32_t b = __float_as_uint(fmaxf(x, 0x1p-126f)) + 0x007fffffu;
  return __uint_as_float(min(b & 0x7f800000u, 0x7e800000u));
}
__device__ __forceinline__ float pow2_inverse(float x) {
  return __uint_as_float(0x7f000000u - __float_as_uint(x));
}
// The largest sum of weights with which a tile's weights, times up to four, fit
// f16, which ends at 65504.
constexpr float kMaxWeights = 8192.0f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four codes -> two f16 pairs, exactly.  int8: u = c + 128 in the low byte of
// 0x6400 is the half 1024 + u.
template <int CODE>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (CODE == KDA_I8) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
    __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    lo = *reinterpret_cast<uint32_t*>(&x);
    hi = *reinterpret_cast<uint32_t*>(&y);
  } else {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n"
        " cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A power of two by which a row of bf16 values with largest magnitude `most`
// (bits, sign off) is divided so that it fits f16: most lands in [1, 2).
// Elements below 2^-14 of it lose bits: 2^-25 of `most` at worst.  Infinity
// and NaN stay what they are.  Returns the exponent.
__device__ __forceinline__ int row_exponent(uint32_t most) {
  const int e = (int)(most >> 23) - 127;
  return most == 0 || most >= 0x7f800000u ? 0 : min(max(e, -126), 126);
}
__device__ __forceinline__ float exp2i(int e) {  // -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

}  // namespace kda_cache

// The kernels for few rows and for tiles of rows, and the join of the parts
// that both have left (`tile`.ctas 0: the tile kernel has not run).  The later
// ones are launched so that their start overlaps the end of the one before.
kda_status kda_launch_attn_rows(const kda_cache::AttnArgs& p, int d, int code, cudaStream_t s);
kda_status kda_launch_attn_tile(const kda_cache::AttnArgs& p, int d, int code, cudaStream_t s);
kda_status kda_launch_attn_join(const kda_cache::AttnArgs& p, const kda_cache::Parts& tile, int d,
                                cudaStream_t s);

namespace kda_cache {

// Programmatic dependent launch: the kernel may start when the one before it
// in the stream has let it (kernel_may_follow), and must call
// wait_for_kernel_before at a point after which it needs, or before it ends
// and so lets others need, what that one wrote.
__device__ __forceinline__ void kernel_may_follow() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_kernel_before() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class... Params, class... Args>
inline kda_status launch_following(void (*kernel)(Params...), dim3 grid, dim3 block, int smem,
                                   cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda_cache
