// kda_cache_attn.cu -- attention of a step's queries over the paged 8-bit
// cache: argument checks and kernels.
#include "kda_cache_attn.cuh"

namespace {

using namespace kda_cache;

size_t r256(size_t x) { return (x + 255) / 256 * 256; }

// Workspace: for the few-row kernel, then (where a request may have more
// rows) for the tile kernel, the batch's units, the CTAs' entered segments
// and their parts.
struct Layout {
  int ctas[2];
  size_t total[2], head[2], ml[2], o[2], bytes;
};
constexpr int kPartRows[2] = {kFewRows, kTileRows};
// (the tile kernel's third: a piece of a long run of key tiles)
constexpr int kPartSlots[2] = {2, 3};

Layout layout(int max_new, int G, int d) {
  Layout w{};
  const int device_sms = kda_device_sms(), sms = device_sms < kMaxSms ? device_sms : kMaxSms;
  const int64_t rows = (int64_t)max_new * G;
  w.ctas[0] = sms * kRowsPerSm;
  w.ctas[1] = rows > few_max(d) ? sms / 2 : 0;  // (pairs of CTAs)
  size_t at = 0;
  for (int i = 0; i < 2; ++i) {
    const size_t parts = (size_t)kPartSlots[i] * w.ctas[i] * kPartRows[i];
    w.total[i] = at;
    w.head[i] = at + 256;
    w.ml[i] = w.head[i] + r256(w.ctas[i] * sizeof(PartHead));
    w.o[i] = w.ml[i] + r256(parts * 8);
    at = w.o[i] + r256(parts * d * 4);
  }
  w.bytes = at;
  return w;
}

// Reports malformed requests of a call that computes nothing.
constexpr int kCheckThreads = 256;
__global__ void __launch_bounds__(kCheckThreads) kda_attn_check_kernel(AttnArgs p) {
  for (int r = blockIdx.x * kCheckThreads + threadIdx.x; r < p.R; r += gridDim.x * kCheckThreads) {
    bool bad;
    load_req(p, r, bad);
    if (bad) report(p.status, KDA_ERR_BAD_SEQLENS);
  }
}

}  // namespace

extern "C" size_t kda_cache_attn_workspace_bytes(int R, int T, int max_new, int Hq, int Hkv,
                                                 int d) {
  if (R < 1 || T < 1 || max_new < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || !head_dim_ok(d)) return 0;
  return layout(max_new, Hq / Hkv, d).bytes;
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
      Hq / Hkv > 64 || Hkv > 4096 || R > kMaxRequests)
    return KDA_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * page > (1 << 30) || T > (1 << 26)) return KDA_ERR_UNSUPPORTED;
  const int64_t width = (int64_t)Hq * d;
  if (q_stride < width) return KDA_ERR_INVALID_ARG;
  if (q_stride % 8 || !aligned(16, q, out, k_codes, v_codes) ||
      !aligned(4, cu_seqlens, kv_lens, block_table, k_scale, v_scale, lse, dev_status))
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
  int lg = 4;
  while ((1 << lg) < page) ++lg;
  AttnArgs p{q, q_stride, cu_seqlens, kv_lens, block_table, (const uint8_t*)k_codes,
             (const uint8_t*)v_codes, k_scale, v_scale, out, lse, dev_status, R, T, max_new,
             max_pages, Hq, Hkv, Hq / Hkv, num_pages, lg, few_max(d), scale, {}};
  if (T == 0 || max_new == 0) {  // (what is new then is more than the caller has rows for)
    if (!dev_status) return KDA_OK;
    kda_attn_check_kernel<<<(R + kCheckThreads - 1) / kCheckThreads, kCheckThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
  }
  const Layout w = layout(max_new, p.G, d);
  if (w.ctas[0] < 1) return KDA_ERR_CUDA;
  const bool own = workspace == nullptr;
  if (own && cudaMallocAsync(&workspace, w.bytes, s) != cudaSuccess) return KDA_ERR_CUDA;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  Parts parts[2];
  for (int i = 0; i < 2; ++i)
    parts[i] = {w.ctas[i], kPartRows[i], reinterpret_cast<int64_t*>(ws + w.total[i]),
                reinterpret_cast<PartHead*>(ws + w.head[i]), reinterpret_cast<float*>(ws + w.ml[i]),
                reinterpret_cast<float*>(ws + w.o[i])};
  p.parts = parts[0];
  kda_status rc = kda_launch_attn_rows(p, d, code, s);
  if (rc == KDA_OK && parts[1].ctas) {
    p.parts = parts[1];
    rc = kda_launch_attn_tile(p, d, code, s);
  }
  p.parts = parts[0];
  if (rc == KDA_OK) rc = kda_launch_attn_join(p, parts[1], d, s);
  if (own && cudaFreeAsync(workspace, s) != cudaSuccess && rc == KDA_OK) rc = KDA_ERR_CUDA;
  return rc;
}
