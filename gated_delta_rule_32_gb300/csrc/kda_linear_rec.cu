// kda_linear_rec.cu -- linear attention with a decay for each head, token by
// token: decode steps, and the prompts of types and head sizes that the
// tensor cores do not serve.
//
//   S <- e^a S + k v^T,   o = scale * S^T q      (S: dk x dv of a sequence and head)
//
// A CTA holds DVB value columns of one S in registers, so S moves through
// memory once a call whatever the number of tokens: a thread has four adjacent
// columns of DK / RG rows, and at each step of its loads the CTA reads
// consecutive 16-byte pieces.  The inputs of TB tokens are fetched into registers
// while the block before is at work (the first while the state is on its way) and
// put into shared memory; then every thread runs its tokens without a barrier,
// leaving each token's sum over its warp's rows in shared memory, and one pass
// adds the warps' parts.
//
// A decode step is bound by the states' bytes: 64 sequences, 32 heads of 128 x
// 128 take 43 us, 6.3 TB/s (inputs fetched after the states: 50 us).  Long runs
// are bound by the chain of tokens, some 180 ns each: 2 rows of 333 tokens, 4
// heads of 64 x 32, fp32, 62 us.
//
// A slow decay's factor is close to 1, and its rounding to 24 bits would be the
// same at every token: 2^-25 times 10 000 tokens is more than the sums' own
// rounding.  So e^a enters as two numbers, 1 + (e^a - 1) and what that lost.
#include "kda_linear.cuh"

namespace {

using namespace kda_linear;

template <typename Tin, int DK, int DVB>
struct Rec {
  static constexpr int kThreads = DK * DVB / 4 < 256 ? DK * DVB / 4 : 256;
  static constexpr int CL = DVB / 4;            // threads across the columns
  static constexpr int RG = kThreads / CL;      // rows read at a time
  static constexpr int R = DK / RG;             // rows of a thread: RG apart
  static constexpr int kWarps = kThreads / 32;
  // tokens at a time, as many as static shared memory has room for (8 instead of 16: 61 us
  // where 16 took 59)
  static constexpr int TB = DVB <= 32 ? 16 : 8;
  static constexpr bool kAsk = DVB <= 32;       // a block asks first whether a token forgets
};

template <typename Tin, int DK, int DVB>
__global__ void __launch_bounds__(Rec<Tin, DK, DVB>::kThreads)
    kda_linear_rec_kernel(const LinearArgs p) {
  using L = Rec<Tin, DK, DVB>;
  constexpr int TB = L::TB;
  __shared__ float s_k[TB][DK], s_q[TB][DK], s_e[TB], s_l[TB];
  __shared__ bool s_some;  // a token of the block forgets
  __shared__ __align__(16) float s_v[TB][DVB], s_o[TB][L::kWarps][DVB];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cb = p.dv / DVB;
  const int unit = blockIdx.x / cb, c0 = (blockIdx.x - unit * cb) * DVB;
  const int n = unit / p.H, h = unit - n * p.H, hk = h / (p.H / p.HK);
  const int rg = tid / L::CL, cl = (tid - rg * L::CL) * 4;
  int64_t row;
  int len;
  if (!span(p, n, row, len)) return;
  const int64_t at = ((int64_t)unit * DK + rg) * p.dv + c0 + cl, step = (int64_t)L::RG * p.dv;
  float4 S[L::R];
#pragma unroll
  for (int r = 0; r < L::R; ++r)
    S[r] = p.init ? *reinterpret_cast<const float4*>(p.init + at + r * step)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
  const Tin* q = static_cast<const Tin*>(p.q) + row * p.q_stride + hk * DK;
  const Tin* k = static_cast<const Tin*>(p.k) + row * p.k_stride + hk * DK;
  const Tin* v = static_cast<const Tin*>(p.v) + row * p.v_stride + (int64_t)h * p.dv + c0;
  const float* a = p.decay + row * p.decay_stride + h;
  Tin* out = static_cast<Tin*>(p.out) + (row * p.H + h) * p.dv + c0;
  // a block's inputs: fetched into registers while the block before is at work
  constexpr int NK = (TB * DK + L::kThreads - 1) / L::kThreads;
  constexpr int NV = (TB * DVB + L::kThreads - 1) / L::kThreads;
  float fk[NK], fq[NK], fv[NV], fa = 0.0f;
  auto fetch = [&](int t0) {
    const int nt = len - t0 < TB ? len - t0 : TB;
#pragma unroll
    for (int x = 0; x < NK; ++x) {
      const int e = tid + x * L::kThreads, t = e / DK, i = e - t * DK;
      if (t < nt) {
        fk[x] = kda::to_f32(k[(t0 + t) * p.k_stride + i]);
        fq[x] = kda::to_f32(q[(t0 + t) * p.q_stride + i]);
      }
    }
#pragma unroll
    for (int x = 0; x < NV; ++x) {
      const int e = tid + x * L::kThreads, t = e / DVB, c = e - t * DVB;
      if (t < nt) fv[x] = kda::to_f32(v[(t0 + t) * p.v_stride + c]);
    }
    if (tid < nt) fa = a[(t0 + tid) * p.decay_stride];
  };
  if (len > 0) fetch(0);
  for (int t0 = 0; t0 < len; t0 += TB) {
    const int nt = len - t0 < TB ? len - t0 : TB;
#pragma unroll
    for (int x = 0; x < NK; ++x) {
      const int e = tid + x * L::kThreads, t = e / DK, i = e - t * DK;
      if (t < nt) {
        s_k[t][i] = fk[x];
        s_q[t][i] = fq[x];
      }
    }
#pragma unroll
    for (int x = 0; x < NV; ++x) {
      const int e = tid + x * L::kThreads, t = e / DVB, c = e - t * DVB;
      if (t < nt) s_v[t][c] = fv[x];
    }
    bool cut = false;
    if (tid < nt) {
      const float x = clamp_decay(fa);
      const float m = expm1f(x), e = 1.0f + m;
      cut = forgets(x);
      s_e[tid] = cut ? -1.0f : x > -0.5f ? e : expf(x);
      s_l[tid] = x > -0.5f ? m - (e - 1.0f) : 0.0f;
    }
    if (L::kAsk && warp == 0) {
      cut = __any_sync(0xffffffffu, cut);
      if (lane == 0) s_some = cut;
    }
    if (t0 + TB < len) fetch(t0 + TB);
    __syncthreads();
    auto step = [&](int t, float e) {
      const float l = s_l[t];
      const float4 vv = *reinterpret_cast<const float4*>(&s_v[t][cl]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < L::R; ++r) {
        const float kk = s_k[t][rg + r * L::RG], qq = s_q[t][rg + r * L::RG];
        S[r].x = fmaf(e, S[r].x, fmaf(l, S[r].x, kk * vv.x));
        S[r].y = fmaf(e, S[r].y, fmaf(l, S[r].y, kk * vv.y));
        S[r].z = fmaf(e, S[r].z, fmaf(l, S[r].z, kk * vv.z));
        S[r].w = fmaf(e, S[r].w, fmaf(l, S[r].w, kk * vv.w));
        o.x = fmaf(qq, S[r].x, o.x);
        o.y = fmaf(qq, S[r].y, o.y);
        o.z = fmaf(qq, S[r].z, o.z);
        o.w = fmaf(qq, S[r].w, o.w);
      }
#pragma unroll
      for (int x = L::CL; x < 32; x *= 2) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
      }
      if (lane < L::CL) *reinterpret_cast<float4*>(&s_o[t][warp][cl]) = o;
    };
    // Narrow blocks are bound by the chain of tokens, where a branch on the token's factor takes
    // time (the case of 62 us above 64): they have it only if one of the block's tokens forgets.
    // Wide ones have it at each token (the decode step takes 2 % more with two loops).
    if (L::kAsk && !s_some) {
      for (int t = 0; t < nt; ++t) step(t, s_e[t]);
    } else {
      for (int t = 0; t < nt; ++t) {
        const float e = s_e[t];
        if (e < 0.0f) {  // (the same for all: what it is multiplied by next is finite)
#pragma unroll
          for (int r = 0; r < L::R; ++r) S[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        step(t, e);
      }
    }
    __syncthreads();
    for (int e = tid; e < nt * DVB; e += L::kThreads) {
      const int t = e / DVB, c = e - t * DVB;
      float o = 0.0f;
#pragma unroll
      for (int w = 0; w < L::kWarps; ++w) o += s_o[t][w][c];
      out[(int64_t)(t0 + t) * p.H * p.dv + c] = kda::from_f32<Tin>(p.scale * o);
    }
  }
  if (p.final_state) {
#pragma unroll
    for (int r = 0; r < L::R; ++r)
      *reinterpret_cast<float4*>(p.final_state + at + r * step) = S[r];
  }
}

template <typename Tin, int DK, int DVB>
void launch(const LinearArgs& p, cudaStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.N * p.H * (p.dv / DVB));
  kda_linear_rec_kernel<Tin, DK, DVB><<<grid, Rec<Tin, DK, DVB>::kThreads, 0, s>>>(p);
}

template <typename Tin, int DK>
void launch_dv(const LinearArgs& p, int dvb, cudaStream_t s) {
  switch (dvb) {
    case 16: launch<Tin, DK, 16>(p, s); break;
    case 32: launch<Tin, DK, 32>(p, s); break;
    case 64: launch<Tin, DK, 64>(p, s); break;
    default: launch<Tin, DK, 128>(p, s); break;
  }
}

template <typename Tin>
void launch_dk(const LinearArgs& p, int dvb, cudaStream_t s) {
  switch (p.dk) {
    case 16: launch_dv<Tin, 16>(p, dvb, s); break;
    case 32: launch_dv<Tin, 32>(p, dvb, s); break;
    case 64: launch_dv<Tin, 64>(p, dvb, s); break;
    default: launch_dv<Tin, 128>(p, dvb, s); break;
  }
}

}  // namespace

kda_status kda_launch_linear_rec(const LinearArgs& p, kda_dtype dtype, cudaStream_t stream) {
  // few (sequence, head) units: their columns over more CTAs
  int dvb = p.dv;
  while (dvb > 32 && (int64_t)p.N * p.H * (p.dv / dvb) < kda_device_sms()) dvb /= 2;
  if (dtype == KDA_F32)
    launch_dk<float>(p, dvb, stream);
  else
    launch_dk<__nv_bfloat16>(p, dvb, stream);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
