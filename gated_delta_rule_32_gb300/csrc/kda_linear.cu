// kda_linear.cu -- linear attention with a decay for each head: argument
// checks and the choice of the kernel.
#include "kda_cache.cuh"
#include "kda_linear.cuh"

namespace {

using namespace kda_linear;
using kda_cache::aligned;
using kda_cache::overlaps;

bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// What a tensor of `rows` rows, `stride` elements apart, spans in bytes.
size_t extent(int64_t rows, int64_t stride, int64_t width, int size) {
  return rows ? (size_t)((rows - 1) * stride + width) * size : 0;
}

// The rules that both entry points share; rows: token rows of the inputs.
kda_status check(const LinearArgs& p, kda_dtype dtype, int64_t rows) {
  if (p.N < 1 || p.T < 0 || p.H < 1 || p.HK < 1 || p.H % p.HK) return KDA_ERR_INVALID_ARG;
  if (rows > 0 && (!p.q || !p.k || !p.v || !p.decay || !p.out)) return KDA_ERR_INVALID_ARG;
  if ((dtype != KDA_BF16 && dtype != KDA_F32) || !dim_ok(p.dk) || !dim_ok(p.dv))
    return KDA_ERR_UNSUPPORTED;
  if (rows > (1 << 30) || p.H > 65536 || (int64_t)p.N * p.H > (1 << 28)) return KDA_ERR_UNSUPPORTED;
  const int64_t kw = (int64_t)p.HK * p.dk, vw = (int64_t)p.H * p.dv;
  if (p.q_stride < kw || p.k_stride < kw || p.v_stride < vw) return KDA_ERR_INVALID_ARG;
  if (p.decay_stride != 0 && p.decay_stride < p.H) return KDA_ERR_INVALID_ARG;
  const int size = dtype == KDA_F32 ? 4 : 2, unit = 16 / size;
  for (int64_t x : {p.q_stride, p.k_stride, p.v_stride, p.decay_stride})
    if (x > ((int64_t)1 << 30)) return KDA_ERR_UNSUPPORTED;
  if (p.q_stride % unit || p.k_stride % unit || p.v_stride % unit) return KDA_ERR_MISALIGNED;
  if (!aligned(16, p.q, p.k, p.v, p.out, p.init, p.final_state) ||
      !aligned(4, p.decay, p.cu, p.status))
    return KDA_ERR_MISALIGNED;
  const size_t out_n = (size_t)rows * vw * size, st_n = (size_t)p.N * p.H * p.dk * p.dv * 4;
  const void* ins[] = {p.q, p.k, p.v, p.decay, p.cu};
  const size_t in_n[] = {extent(rows, p.q_stride, kw, size), extent(rows, p.k_stride, kw, size),
                         extent(rows, p.v_stride, vw, size),
                         rows ? extent(p.decay_stride ? rows : 1, p.decay_stride, p.H, 4) : 0,
                         (size_t)(p.N + 1) * 4};
  for (int i = 0; i < 5; ++i)
    if (overlaps(p.out, out_n, ins[i], in_n[i]) || overlaps(p.final_state, st_n, ins[i], in_n[i]))
      return KDA_ERR_INVALID_ARG;
  if (overlaps(p.out, out_n, p.init, st_n) || overlaps(p.out, out_n, p.final_state, st_n))
    return KDA_ERR_INVALID_ARG;
  if (p.init != p.final_state && overlaps(p.init, st_n, p.final_state, st_n))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

}  // namespace

extern "C" size_t kda_linear_workspace_bytes(int B, int T, int H, int dk, int dv, kda_dtype dtype,
                                             int packed) {
  if (B < 1 || T < 1 || H < 1 || !kda_linear_tile_ok(dk, dv, dtype)) return 0;
  if (H > 65536 || (int64_t)B * H > (1 << 28)) return 0;
  return kda_linear_tile_workspace(B, T, H, dk, dv, packed != 0);
}

extern "C" kda_status kda_linear_fwd(const void* q, int64_t q_stride, const void* k,
                                     int64_t k_stride, const void* v, int64_t v_stride,
                                     const float* log_decay, int64_t decay_stride,
                                     const float* init_state, void* out, float* final_state,
                                     int B, int T, int H, int Hk, int dk, int dv,
                                     const int32_t* cu_seqlens, kda_dtype dtype, float scale,
                                     void* workspace, size_t workspace_bytes,
                                     int32_t* dev_status, kda_stream_t stream) {
  const LinearArgs p{q, k, v, q_stride, k_stride, v_stride, log_decay, decay_stride, init_state,
                     out, final_state, cu_seqlens, dev_status, B, T, H, Hk, dk, dv, scale};
  const kda_status rc = check(p, dtype, cu_seqlens ? T : (int64_t)B * T);
  if (rc != KDA_OK) return rc;
  const size_t need = kda_linear_workspace_bytes(B, T, H, dk, dv, dtype, cu_seqlens != nullptr);
  if (workspace) {
    if (!aligned(256, workspace)) return KDA_ERR_MISALIGNED;
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dev_status && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess)
    return KDA_ERR_CUDA;
  // (without rows the tensor maps have nothing to describe: states only)
  if (T == 0 || !kda_linear_tile_ok(dk, dv, dtype)) return kda_launch_linear_rec(p, dtype, s);
  const bool own = need > 0 && workspace == nullptr;
  if (own && cudaMallocAsync(&workspace, need, s) != cudaSuccess) return KDA_ERR_CUDA;
  kda_status r = kda_launch_linear_tile(p, workspace, s);
  if (own && cudaFreeAsync(workspace, s) != cudaSuccess && r == KDA_OK) r = KDA_ERR_CUDA;
  return r;
}

extern "C" kda_status kda_linear_decode(const void* q, int64_t q_stride, const void* k,
                                        int64_t k_stride, const void* v, int64_t v_stride,
                                        const float* log_decay, int64_t decay_stride, float* state,
                                        void* out, int N, int T, int H, int Hk, int dk, int dv,
                                        kda_dtype dtype, float scale, kda_stream_t stream) {
  if (!state) return KDA_ERR_INVALID_ARG;
  const LinearArgs p{q, k, v, q_stride, k_stride, v_stride, log_decay, decay_stride, state, out,
                     state, nullptr, nullptr, N, T, H, Hk, dk, dv, scale};
  const kda_status rc = check(p, dtype, (int64_t)N * T);
  if (rc != KDA_OK || T == 0) return rc;
  return kda_launch_linear_rec(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}
