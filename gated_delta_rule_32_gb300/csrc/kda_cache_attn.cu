// kda_cache_attn.cu -- attention of a step's queries over the paged 8-bit
// cache: argument checks and kernels.
#include "kda_cache_attn.cuh"

namespace {

using namespace kda_cache;

// The plain form on the GPU: one warp per query row, one key at a time, the
// running maximum and sum of the softmax in fp32.
template <int CODE, int D>
__global__ void __launch_bounds__(128) kda_cache_attn_row_kernel(AttnArgs p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (int64_t)p.T * p.Hq) return;
  const int t = (int)(row / p.Hq), hq = (int)(row % p.Hq), h = hq / p.G;
  int r = -1;
  for (int i = 0; i < p.R; ++i) {
    if (p.cu[i] <= t && t < p.cu[i + 1]) r = i;
    if (p.cu[i + 1] < p.cu[i] && lane == 0) report(p.status, KDA_ERR_BAD_SEQLENS);
  }
  if (r < 0) return;
  const int P = 1 << p.page_log2;
  const int c0 = p.cu[r], n = p.cu[r + 1] - c0, kv = p.kv_lens[r];
  if (n > p.max_new || c0 < 0 || c0 + n > p.T || kv < 0 ||
      kv > ((int64_t)p.max_pages << p.page_log2)) {
    if (lane == 0) report(p.status, KDA_ERR_BAD_SEQLENS);
    return;
  }
  if ((int64_t)n * p.G <= kFewRows) return;
  constexpr int E = D / 32;
  float q[E], o[E] = {};
  for (int e = 0; e < E; ++e)
    q[e] = __uint_as_float((uint32_t)p.q[t * p.q_stride + hq * D + lane * E + e] << 16) * p.scale;
  float m = -INFINITY, l = 0;
  const int seen = min(kv, kv - n + (t - c0) + 1);
  for (int j = 0; j < seen; ++j) {
    const int pg = p.table[(int64_t)r * p.max_pages + (j >> p.page_log2)];
    if (pg < 0 || pg >= p.num_pages) {
      if (lane == 0) report(p.status, KDA_ERR_BAD_PAGES);
      return;
    }
    const int64_t ph = (int64_t)pg * p.Hkv + h;
    const int64_t at = ((ph << p.page_log2) + (j & (P - 1))) * D + lane * E;
    float s = 0;
    for (int e = 0; e < E; ++e) s += q[e] * decode1<CODE>(p.k_codes[at + e]);
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    s *= p.k_scale[ph] / code_top(CODE);
    const float m1 = fmaxf(m, s), c = expf(m - m1), w = expf(s - m1);
    l = l * c + w;
    m = m1;
    const float wv = w * (p.v_scale[ph] / code_top(CODE));
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + wv * decode1<CODE>(p.v_codes[at + e]);
  }
  for (int e = 0; e < E; ++e)
    reinterpret_cast<__nv_bfloat16*>(p.out)[row * D + lane * E + e] =
        __float2bfloat16_rn(seen > 0 ? o[e] / l : 0.0f);
  if (p.lse && lane == 0) p.lse[row] = seen > 0 ? m + logf(l) : -INFINITY;
}

size_t r256(size_t x) { return (x + 255) / 256 * 256; }

// Workspace: the schedule's prefix sums, then the parts of the few-row kernel
// (two for each of its CTAs).
struct Layout {
  int ctas;
  size_t ml, o, bytes;
};
Layout layout(int R, int max_new, int G, int d) {
  Layout w;
  w.ctas = kda_device_sms() * ((int64_t)max_new * G <= 8 ? 4 : 3);
  w.ml = r256((size_t)(R + 1) * 8);
  w.o = w.ml + r256((size_t)2 * w.ctas * kFewRows * 8);
  w.bytes = w.o + r256((size_t)2 * w.ctas * kFewRows * d * 4);
  return w;
}

}  // namespace

extern "C" size_t kda_cache_attn_workspace_bytes(int R, int T, int max_new, int Hq, int Hkv,
                                                 int d) {
  if (R < 1 || T < 1 || max_new < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || !head_dim_ok(d)) return 0;
  return layout(R, max_new, Hq / Hkv, d).bytes;
}

extern "C" kda_status kda_cache_attn(const uint16_t* q, int64_t q_stride,
                                     const int32_t* cu_seqlens, const int32_t* kv_lens,
                                     const int32_t* block_table, int max_pages,
                                     const void* k_codes, const void* v_codes,
                                     const float* k_scale, const float* v_scale, uint16_t* out,
                                     float* lse, int R, int T, int max_new, int Hq, int Hkv,
                                     int d, int num_pages, int page, kda_code code, float scale,
                                     void* workspace, size_t workspace_bytes,
                                     int32_t* dev_status, kda_stream_t stream) {
  if (R < 1 || T < 0 || max_new < 0 || Hq < 1 || Hkv < 1 || max_pages < 1 || num_pages < 1)
    return KDA_ERR_INVALID_ARG;
  if (!cu_seqlens || !kv_lens || !block_table || !k_codes || !v_codes || !k_scale || !v_scale)
    return KDA_ERR_INVALID_ARG;
  if (T > 0 && (!q || !out)) return KDA_ERR_INVALID_ARG;
  if (Hq % Hkv) return KDA_ERR_INVALID_ARG;
  if (!page_ok(page) || !head_dim_ok(d) || (code != KDA_I8 && code != KDA_E4M3) ||
      Hq / Hkv > 64 || R > kMaxRequests)
    return KDA_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * page > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  const int64_t width = (int64_t)Hq * d;
  if (q_stride < width) return KDA_ERR_INVALID_ARG;
  if (q_stride % 8 || (((uintptr_t)q | (uintptr_t)out | (uintptr_t)k_codes |
                        (uintptr_t)v_codes) & 15) != 0)
    return KDA_ERR_MISALIGNED;
  const size_t pool = (size_t)num_pages * Hkv * page * d, sc = (size_t)num_pages * Hkv * 4;
  const size_t out_n = (size_t)T * width * 2, lse_n = (size_t)T * Hq * 4;
  const void* ins[] = {q, cu_seqlens, kv_lens, block_table, k_codes, v_codes, k_scale, v_scale};
  const size_t in_n[] = {T ? (size_t)((T - 1) * q_stride + width) * 2 : 0, (size_t)(R + 1) * 4,
                         (size_t)R * 4, (size_t)R * max_pages * 4, pool, pool, sc, sc};
  for (int i = 0; i < 8; ++i)
    if (overlaps(out, out_n, ins[i], in_n[i]) || overlaps(lse, lse_n, ins[i], in_n[i]))
      return KDA_ERR_INVALID_ARG;
  if (overlaps(out, out_n, lse, lse_n)) return KDA_ERR_INVALID_ARG;
  if (workspace) {
    if (((uintptr_t)workspace & 255) != 0) return KDA_ERR_MISALIGNED;
    if (workspace_bytes < kda_cache_attn_workspace_bytes(R, T, max_new, Hq, Hkv, d))
      return KDA_ERR_WORKSPACE;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dev_status && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess)
    return KDA_ERR_CUDA;
  if (T == 0 || max_new == 0) return KDA_OK;
  int lg = 4;
  while ((1 << lg) < page) ++lg;
  AttnArgs p{q, q_stride, cu_seqlens, kv_lens, block_table, (const uint8_t*)k_codes,
             (const uint8_t*)v_codes, k_scale, v_scale, out, lse, dev_status, R, T, max_new,
             max_pages, Hq, Hkv, Hq / Hkv, num_pages, lg, scale, nullptr, nullptr, nullptr};
  const Layout w = layout(R, max_new, p.G, d);
  if (w.ctas < 1) return KDA_ERR_CUDA;
  const bool own = workspace == nullptr;
  if (own) {
    if (cudaMallocAsync(&workspace, w.bytes, s) != cudaSuccess) return KDA_ERR_CUDA;
  }
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.prefix = reinterpret_cast<int64_t*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + w.ml);
  p.part_o = reinterpret_cast<float*>(ws + w.o);
  kda_status rc = kda_launch_attn_rows(p, d, code, w.ctas, s);
  if (rc == KDA_OK && (int64_t)max_new * p.G > kFewRows) {
    const unsigned grid = (unsigned)(((int64_t)T * Hq + 3) / 4);
    if (code == KDA_I8) {
      if (d == 64) kda_cache_attn_row_kernel<KDA_I8, 64><<<grid, 128, 0, s>>>(p);
      else kda_cache_attn_row_kernel<KDA_I8, 128><<<grid, 128, 0, s>>>(p);
    } else {
      if (d == 64) kda_cache_attn_row_kernel<KDA_E4M3, 64><<<grid, 128, 0, s>>>(p);
      else kda_cache_attn_row_kernel<KDA_E4M3, 128><<<grid, 128, 0, s>>>(p);
    }
    if (cudaGetLastError() != cudaSuccess) rc = KDA_ERR_CUDA;
  }
  if (own && cudaFreeAsync(workspace, s) != cudaSuccess && rc == KDA_OK) rc = KDA_ERR_CUDA;
  return rc;
}
