// kda_rotary.cu -- rotary positions of a step's queries and keys.
//
// Pair i of a head's first `part` channels is turned by t = position * f_i
// (or -t): (x, y) -> amplitude * (x cos t - y sin t, x sin t + y cos t).
// The angle is taken in whole turns as a 64-bit fraction: f / 2 pi times 2^64
// as an integer times the position, modulo 2^64, with no reduction of large
// angles; sincospif takes it in half turns.  The quotient is formed in two parts
// (one 64-bit floating point number of it would err by up to 2^-54 of itself, times
// the position: 2^-18 of a turn at positions near 2^31 and 100 radians a token) and
// errs by 2^-64 of a turn each: at most 2^-32 of one at any 31-bit position.  That is
// a dozen 64-bit floating point operations, slow here, so a CTA does it once for each
// frequency and its threads read the integers from shared memory.
//
// A thread turns eight pairs of one token in up to eight heads (fewer where the
// batch is small): their sines and cosines are taken once and stay in registers,
// and the loads of four heads go out together.  Memory bound: 37 000 tokens of 32
// + 8 heads of 128 channels take 123 us, 6.2 TB/s read and written; 64 tokens take
// 4.0 us, all of it latency.
#include <type_traits>

#include "kda_cache.cuh"
#include "kda_common.cuh"

namespace {

using kda_cache::aligned;

constexpr int kThreads = 256;

struct RotaryArgs {
  const void* in[2];
  void* out[2];
  int64_t in_stride[2], out_stride[2];  // elements between tokens
  int heads[2], groups[2];              // groups: of `run` heads, the last may be short
  const int32_t* pos;
  const double* freq;
  int T, d, part, run, inverse;
  float amplitude;
};

template <typename T> struct Vec;  // eight channels
template <> struct Vec<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(r[i] << 16);
      x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void put(const float* x) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      r[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    w = make_uint4(r[0], r[1], r[2], r[3]);
  }
};
template <> struct Vec<float> {
  float4 w[2];
  __device__ __forceinline__ void get(float* x) const {
    *reinterpret_cast<float4*>(x) = w[0];
    *reinterpret_cast<float4*>(x + 4) = w[1];
  }
  __device__ __forceinline__ void put(const float* x) {
    w[0] = make_float4(x[0], x[1], x[2], x[3]);
    w[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};
template <typename T>
__device__ __forceinline__ Vec<T> load8(const T* p) {
  Vec<T> v;
  if constexpr (std::is_same<T, float>::value) {
    v.w[0] = reinterpret_cast<const float4*>(p)[0];
    v.w[1] = reinterpret_cast<const float4*>(p)[1];
  } else {
    v.w = *reinterpret_cast<const uint4*>(p);
  }
  return v;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Vec<T>& v) {
  if constexpr (std::is_same<T, float>::value) {
    reinterpret_cast<float4*>(p)[0] = v.w[0];
    reinterpret_cast<float4*>(p)[1] = v.w[1];
  } else {
    *reinterpret_cast<uint4*>(p) = v.w;
  }
}

// What a token turns at f radians, in units of 2^-64 of a turn.
__device__ __forceinline__ uint64_t turn_of(double f) {
  // 1 / 2 pi to some 107 bits
  constexpr double c = 0.15915494309189535, c_lo = -9.839338337591243e-18;
  const double hi = f * c, lo = fma(f, c_lo, fma(f, c, -hi));
  return (uint64_t)__double2ll_rn((hi - rint(hi)) * 18446744073709551616.0) +
         (uint64_t)__double2ll_rn((lo - rint(lo)) * 18446744073709551616.0);
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads) kda_rotary_kernel(const RotaryArgs p) {
  __shared__ __align__(16) uint64_t s_turn[256];  // (d is at most 512)
  __shared__ __align__(16) float s_amplitude[256];
  for (int i = threadIdx.x; i < p.part / 2; i += kThreads) {
    const double f = p.freq[i];
    s_turn[i] = turn_of(f);
    // (integers have no NaN: what a frequency that is no number turns gets one here)
    s_amplitude[i] = isfinite(f) ? p.amplitude : __int_as_float(0x7fffffff);
  }
  __syncthreads();
  // a unit: 16 channels of a head (eight pairs, or two pieces to copy)
  const int units = p.d / 16;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t t = id / units;
  const int u = (int)(id - t * units);
  if (t >= p.T) return;
  const int pos = p.pos[t];
  if (pos < 0) return;
  const int which = (int)blockIdx.y >= p.groups[0];
  const int h0 = ((int)blockIdx.y - (which ? p.groups[0] : 0)) * p.run;
  const int h1 = h0 + p.run < p.heads[which] ? h0 + p.run : p.heads[which];
  const T* in = static_cast<const T*>(p.in[which]) + t * p.in_stride[which];
  T* out = static_cast<T*>(p.out[which]) + t * p.out_stride[which];
  if (16 * u >= p.part) {  // channels without a position
    if (in == out) return;
    for (int h = h0; h < h1; ++h) {
      const int64_t o = (int64_t)h * p.d + 16 * u;
      store8(out + o, load8(in + o));
      store8(out + o + 8, load8(in + o + 8));
    }
    return;
  }
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t turn = s_turn[8 * u + i] * (uint64_t)(uint32_t)pos;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s[i], &c[i]);
    const float amplitude = s_amplitude[8 * u + i];
    c[i] *= amplitude;
    s[i] *= p.inverse ? -amplitude : amplitude;
  }
  const int a = INTER ? 16 * u : 8 * u, b = INTER ? a + 8 : p.part / 2 + 8 * u;
  // (the loads of several heads before their first store)
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;
  for (int h = h0; h < h1; h += kBatch) {
    Vec<T> va[kBatch], vb[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (h + k < h1) {
        const int64_t o = (int64_t)(h + k) * p.d;
        va[k] = load8(in + o + a);
        vb[k] = load8(in + o + b);
      }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (h + k < h1) {
        const int64_t o = (int64_t)(h + k) * p.d;
        float x[16];
        va[k].get(x);
        vb[k].get(x + 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + 8;
          const float xa = x[ia], xb = x[ib];
          x[ia] = xa * c[i] - xb * s[i];
          x[ib] = xa * s[i] + xb * c[i];
        }
        va[k].put(x);
        vb[k].put(x + 8);
        store8(out + o + a, va[k]);
        store8(out + o + b, vb[k]);
      }
  }
}

// `n` rows of `w` bytes, `s` bytes apart.
struct Rows {
  const void* at;
  int64_t s, w, n;
};

// Whether two such sets share a byte; rows of one distance may lie between
// each other.
bool share(const Rows& a, const Rows& b) {
  if (!a.at || !b.at || a.n < 1 || b.n < 1) return false;
  const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
  if (x >= y + (uintptr_t)((b.n - 1) * b.s + b.w) || y >= x + (uintptr_t)((a.n - 1) * a.s + a.w))
    return false;
  if (a.s != b.s) return true;
  const int64_t d = x <= y ? (int64_t)((y - x) % (uintptr_t)a.s)
                           : (a.s - (int64_t)((x - y) % (uintptr_t)a.s)) % a.s;
  return d < a.w || a.s - d < b.w;
}

template <typename T>
void launch(const RotaryArgs& p, bool inter, dim3 grid, cudaStream_t s) {
  if (inter)
    kda_rotary_kernel<T, true><<<grid, kThreads, 0, s>>>(p);
  else
    kda_rotary_kernel<T, false><<<grid, kThreads, 0, s>>>(p);
}

}  // namespace

extern "C" kda_status kda_rotary(const void* q, int64_t q_stride, void* q_out,
                                 int64_t q_out_stride, const void* k, int64_t k_stride,
                                 void* k_out, int64_t k_out_stride, const int32_t* positions,
                                 const double* frequencies, int T, int Hq, int Hk, int d,
                                 int part, float amplitude, int interleaved, int inverse,
                                 kda_dtype dtype, kda_stream_t stream) {
  if (T < 0 || Hq < 0 || Hk < 0 || Hq + Hk < 1 || d < 1 || part < 1 || part > d)
    return KDA_ERR_INVALID_ARG;
  if (T > 0 && (!positions || !frequencies || (Hq && (!q || !q_out)) || (Hk && (!k || !k_out))))
    return KDA_ERR_INVALID_ARG;
  if ((dtype != KDA_BF16 && dtype != KDA_F32) || d % 16 || part % 16 || d > 512 || Hq > 16384 ||
      Hk > 16384 || T > (1 << 30))
    return KDA_ERR_UNSUPPORTED;
  const int size = dtype == KDA_F32 ? 4 : 2, unit = 16 / size;
  RotaryArgs p{{q, k}, {q_out, k_out}, {q_stride, k_stride}, {q_out_stride, k_out_stride},
               {Hq, Hk}, {}, positions, frequencies, T, d, part, 0, inverse, amplitude};
  if (!aligned(16, q, q_out, k, k_out) || !aligned(8, frequencies) || !aligned(4, positions))
    return KDA_ERR_MISALIGNED;
  for (int i = 0; i < 2; ++i) {
    if (!p.heads[i]) continue;
    const int64_t w = (int64_t)p.heads[i] * d;
    if (p.in_stride[i] < w || p.out_stride[i] < w) return KDA_ERR_INVALID_ARG;
    if (p.in_stride[i] > ((int64_t)1 << 30) || p.out_stride[i] > ((int64_t)1 << 30))
      return KDA_ERR_UNSUPPORTED;
    if (p.in_stride[i] % unit || p.out_stride[i] % unit) return KDA_ERR_MISALIGNED;
  }
  // an output is its own input in place, or shares nothing with anything
  Rows in[2], out[2];
  for (int i = 0; i < 2; ++i) {
    const int64_t w = (int64_t)p.heads[i] * d * size, n = p.heads[i] ? T : 0;
    in[i] = {p.in[i], p.in_stride[i] * size, w, n};
    out[i] = {p.out[i], p.out_stride[i] * size, w, n};
  }
  for (int i = 0; i < 2; ++i) {
    if (share(out[i], {positions, 4, 4, T}) || share(out[i], {frequencies, 8, 8, part / 2}))
      return KDA_ERR_INVALID_ARG;
    for (int j = 0; j < 2; ++j) {
      const bool place = i == j && in[i].at == out[i].at && in[i].s == out[i].s;
      if (!place && share(out[i], in[j])) return KDA_ERR_INVALID_ARG;
    }
  }
  if (share(out[0], out[1])) return KDA_ERR_INVALID_ARG;
  if (T == 0) return KDA_OK;
  const int64_t blocks = ((int64_t)T * (d / 16) + kThreads - 1) / kThreads;
  p.run = 1;
  while (p.run < 8 && blocks * (Hq + Hk) / (2 * p.run) >= 8 * kda_device_sms()) p.run *= 2;
  for (int i = 0; i < 2; ++i) p.groups[i] = (p.heads[i] + p.run - 1) / p.run;
  const dim3 grid((unsigned)blocks, (unsigned)(p.groups[0] + p.groups[1]));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == KDA_F32)
    launch<float>(p, interleaved != 0, grid, s);
  else
    launch<__nv_bfloat16>(p, interleaved != 0, grid, s);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
