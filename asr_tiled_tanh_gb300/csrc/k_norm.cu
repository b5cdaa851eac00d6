// k_norm.cu -- group norm with an activation over encoder frames, channels
// last (include/rnnt_ops.h).
#include "ops.h"

namespace rnnt {
namespace {

struct NormArgs {
  int B, T, C, G, cg, act;
  float eps;
  long long xf, xb, yf, yb;
  const float* gamma;
  const float* beta;
  const int32_t* T_len;
  float2* stats;  // (mean, rstd) [B,G]
  int32_t* status;
};

__device__ __forceinline__ int frames_of(const NormArgs& a, int b) {
  if (!a.T_len) return a.T;
  const int t = __ldg(a.T_len + b);
  if (t < 0 || t > a.T) {
    report(a.status, RNNT_ERR_LENGTH_RANGE);
    return 0;
  }
  return t;
}

__device__ __forceinline__ float sigmoid_f(float u) { return 1.f / (1.f + expf(-u)); }

__device__ __forceinline__ float act_f(int act, float u) {
  if (act == RNNT_ACT_SILU) return u * sigmoid_f(u);
  if (act == RNNT_ACT_RELU) return u < 0.f ? 0.f : u;  // (NaN stays NaN)
  return u;
}
__device__ __forceinline__ float dact_f(int act, float u) {
  if (act == RNNT_ACT_SILU) {
    const float s = sigmoid_f(u);
    return s * (1.f + u * (1.f - s));
  }
  if (act == RNNT_ACT_RELU) return u > 0.f ? 1.f : 0.f;
  return 1.f;
}

// Sum over the block (256 threads), the same value in every thread.
__device__ float block_sum(float v) {
  __shared__ float part[9];
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < 8; ++i) s += part[i];
  return s;
}

// One block per sample and group.
template <typename T>
__global__ void __launch_bounds__(256)
k_norm_fwd(NormArgs a, const T* __restrict__ x, T* __restrict__ y) {
  const int b = blockIdx.x / a.G, g = blockIdx.x - b * a.G;
  const int tb = frames_of(a, b);
  const long long n = (long long)tb * a.cg;
  const T* xs = x + b * a.xb + (long long)g * a.cg;
  T* ys = y + b * a.yb + (long long)g * a.cg;
  float s = 0.f;
  for (long long i = threadIdx.x; i < n; i += 256) s += to_f<T>(xs[i / a.cg * a.xf + i % a.cg]);
  const float mean = n ? block_sum(s) / (float)n : 0.f;
  float q = 0.f;
  for (long long i = threadIdx.x; i < n; i += 256) {
    const float d = to_f<T>(xs[i / a.cg * a.xf + i % a.cg]) - mean;
    q += d * d;
  }
  const float rstd = n ? rsqrtf(block_sum(q) / (float)n + a.eps) : 0.f;
  if (threadIdx.x == 0) a.stats[blockIdx.x] = make_float2(mean, rstd);
  for (long long i = threadIdx.x; i < (long long)a.T * a.cg; i += 256) {
    const long long t = i / a.cg;
    const int c = (int)(i % a.cg), ch = g * a.cg + c;
    float v = 0.f;
    if (t < tb) {
      const float xh = (to_f<T>(xs[t * a.xf + c]) - mean) * rstd;
      v = act_f(a.act, xh * (a.gamma ? a.gamma[ch] : 1.f) + (a.beta ? a.beta[ch] : 0.f));
    }
    ys[t * a.yf + c] = from_f<T>(v);
  }
}

// One block per sample and group; part: per sample and channel (sum g xh, sum g).
template <typename T>
__global__ void __launch_bounds__(256)
k_norm_bwd(NormArgs a, const T* __restrict__ x, const T* __restrict__ dy, T* __restrict__ dx,
           float2* __restrict__ part) {
  const int b = blockIdx.x / a.G, g = blockIdx.x - b * a.G;
  const int tb = frames_of(a, b);
  const T* xs = x + b * a.xb + (long long)g * a.cg;
  const T* dys = dy + b * a.yb + (long long)g * a.cg;
  T* dxs = dx + b * a.xb + (long long)g * a.cg;
  const float2 st = a.stats[blockIdx.x];
  float m1 = 0.f, m2 = 0.f;
  for (int c = 0; c < a.cg; ++c) {
    const int ch = g * a.cg + c;
    const float ga = a.gamma ? a.gamma[ch] : 1.f, be = a.beta ? a.beta[ch] : 0.f;
    float s1 = 0.f, s2 = 0.f;
    for (int t = threadIdx.x; t < tb; t += 256) {
      const float xh = (to_f<T>(xs[t * a.xf + c]) - st.x) * st.y;
      const float gg = __fmul_rn(to_f<T>(dys[t * a.yf + c]), dact_f(a.act, xh * ga + be));
      s1 += gg;
      s2 += gg * xh;
    }
    s1 = block_sum(s1);
    s2 = block_sum(s2);
    if (threadIdx.x == 0) part[(long long)b * a.C + ch] = make_float2(s2, s1);
    m1 = fmaf(ga, s1, m1);
    m2 = fmaf(ga, s2, m2);
  }
  const long long n = (long long)tb * a.cg;
  if (n) { m1 /= (float)n; m2 /= (float)n; }
  for (long long i = threadIdx.x; i < (long long)a.T * a.cg; i += 256) {
    const long long t = i / a.cg;
    const int c = (int)(i % a.cg), ch = g * a.cg + c;
    float v = 0.f;
    if (t < tb) {
      const float ga = a.gamma ? a.gamma[ch] : 1.f, be = a.beta ? a.beta[ch] : 0.f;
      const float xh = (to_f<T>(xs[t * a.xf + c]) - st.x) * st.y;
      const float gg = __fmul_rn(to_f<T>(dys[t * a.yf + c]), dact_f(a.act, xh * ga + be));
      v = st.y * (fmaf(gg, ga, -m1) - xh * m2);
    }
    dxs[t * a.xf + c] = from_f<T>(v);
  }
}

__global__ void __launch_bounds__(256)
k_norm_params(const float2* __restrict__ part, int B, int C, float* __restrict__ dgamma,
              float* __restrict__ dbeta) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= C) return;
  float s = 0.f, q = 0.f;
  for (int b = 0; b < B; ++b) {
    const float2 p = part[(long long)b * C + c];
    s += p.x;
    q += p.y;
  }
  if (dgamma) dgamma[c] = s;
  if (dbeta) dbeta[c] = q;
}

bool norm_args(const rnnt_norm_dims* d, NormArgs* a) {
  if (!d || d->B < 0 || d->T < 1 || d->C < 1 || d->G < 1 || d->C % d->G) return false;
  if (d->T > (1 << 20) || (long long)d->B * d->G > (1LL << 27)) return false;
  if (d->act < RNNT_ACT_NONE || d->act > RNNT_ACT_RELU || !op_dtype(d->dtype)) return false;
  if (!(d->eps >= 0.f)) return false;
  a->B = d->B; a->T = d->T; a->C = d->C; a->G = d->G; a->cg = d->C / d->G;
  a->act = d->act; a->eps = d->eps;
  a->xf = d->x_frame ? d->x_frame : d->C;
  a->xb = d->x_batch ? d->x_batch : d->T * a->xf;
  a->yf = d->y_frame ? d->y_frame : d->C;
  a->yb = d->y_batch ? d->y_batch : d->T * a->yf;
  // frames and samples must not overlap (outputs use the same strides)
  return a->xf >= d->C && a->yf >= d->C && a->xb >= (d->T - 1) * a->xf + d->C &&
         a->yb >= (d->T - 1) * a->yf + d->C;
}

rnnt_status norm_check(const rnnt_norm_dims* d, NormArgs* a, const void* x, const void* y,
                       const void* saved, const void* ws, size_t ws_bytes, const float* gamma,
                       const float* beta, const int32_t* T_len, int32_t* status) {
  if (!norm_args(d, a)) return RNNT_ERR_INVALID_ARG;
  if (a->B > 0 && (!x || !y || !saved)) return RNNT_ERR_INVALID_ARG;
  const int e = op_size(d->dtype);
  if (!ws || !aligned_to(ws, ALIGN) || !aligned_to(saved, ALIGN) || !aligned_to(x, e) ||
      !aligned_to(y, e) || !aligned_to(gamma, 4) || !aligned_to(beta, 4) ||
      !aligned_to(T_len, 4) || !aligned_to(status, 4))
    return RNNT_ERR_INVALID_ARG;
  if (ws_bytes < rnnt_norm_workspace_bytes(d)) return RNNT_ERR_WORKSPACE_TOO_SMALL;
  a->gamma = gamma; a->beta = beta; a->T_len = T_len; a->status = status;
  a->stats = (float2*)saved;
  return RNNT_OK;
}

}  // namespace
}  // namespace rnnt

using namespace rnnt;

extern "C" {

size_t rnnt_norm_saved_bytes(const rnnt_norm_dims* dims) {
  NormArgs a;
  return norm_args(dims, &a) ? align_up(8 * (size_t)a.B * a.G + 8) : 0;
}

size_t rnnt_norm_workspace_bytes(const rnnt_norm_dims* dims) {
  NormArgs a;
  return norm_args(dims, &a) ? align_up(8 * (size_t)a.B * a.C + 8) : 0;
}

rnnt_status rnnt_norm_fwd(const rnnt_norm_dims* dims, const void* x, const float* gamma,
                          const float* beta, const int32_t* T_len, void* y, void* saved, void* ws,
                          size_t ws_bytes, int32_t* status, rnnt_stream stream) {
  NormArgs a;
  const rnnt_status s =
      norm_check(dims, &a, x, y, saved, ws, ws_bytes, gamma, beta, T_len, status);
  if (s != RNNT_OK) return s;
  if (a.B == 0) return RNNT_OK;
  cudaStream_t st = (cudaStream_t)stream;
  ProfScope ps("norm_fwd", st);
  if (dims->dtype == RNNT_F32)
    k_norm_fwd<<<a.B * a.G, 256, 0, st>>>(a, (const float*)x, (float*)y);
  else
    k_norm_fwd<<<a.B * a.G, 256, 0, st>>>(a, (const __nv_bfloat16*)x, (__nv_bfloat16*)y);
  OPS_CHECK(cudaGetLastError());
  return RNNT_OK;
}

rnnt_status rnnt_norm_bwd(const rnnt_norm_dims* dims, const void* x, const void* dy,
                          const float* gamma, const float* beta, const int32_t* T_len,
                          const void* saved, void* dx, float* dgamma, float* dbeta, void* ws,
                          size_t ws_bytes, int32_t* status, rnnt_stream stream) {
  NormArgs a;
  const rnnt_status s =
      norm_check(dims, &a, x, dy, saved, ws, ws_bytes, gamma, beta, T_len, status);
  if (s != RNNT_OK) return s;
  if (a.B > 0 && !dx) return RNNT_ERR_INVALID_ARG;
  if (!aligned_to(dx, op_size(dims->dtype)) || !aligned_to(dgamma, 4) || !aligned_to(dbeta, 4))
    return RNNT_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  float2* part = (float2*)ws;
  if (a.B > 0) {
    ProfScope ps("norm_bwd", st);
    if (dims->dtype == RNNT_F32)
      k_norm_bwd<<<a.B * a.G, 256, 0, st>>>(a, (const float*)x, (const float*)dy, (float*)dx,
                                            part);
    else
      k_norm_bwd<<<a.B * a.G, 256, 0, st>>>(a, (const __nv_bfloat16*)x, (const __nv_bfloat16*)dy,
                                            (__nv_bfloat16*)dx, part);
    OPS_CHECK(cudaGetLastError());
  }
  ProfScope ps("norm_params", st);
  k_norm_params<<<(int)cdiv(a.C, 256), 256, 0, st>>>(part, a.B, a.C, dgamma, dbeta);
  OPS_CHECK(cudaGetLastError());
  return RNNT_OK;
}

}  // extern "C"
