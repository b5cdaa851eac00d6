// k_orth.cu -- orthogonalised update by Newton-Schulz products
// (include/rnnt_ops.h).
#include "ops.h"

namespace rnnt {
namespace {

// The Muon optimiser's quintic.
constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;

template <typename T>
__global__ void __launch_bounds__(1024)
k_orth_norm(const T* __restrict__ G, int R, int K, long long ld, float eps, float* out) {
  __shared__ double part[32];
  double s = 0;
  for (long long i = threadIdx.x; i < (long long)R * K; i += 1024) {
    const float v = to_f<T>(G[i / K * ld + i % K]);
    s += (double)v * v;
  }
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0;
    for (int i = 0; i < 32; ++i) s += part[i];
    // (a norm that is not finite makes the whole matrix NaN, not 0)
    *out = isfinite(s) ? 1.f / ((float)sqrt(s) + eps) : __int_as_float(0x7fc00000);
  }
}

template <typename T>
__global__ void k_orth_scale(const T* __restrict__ G, int R, int K, long long ld,
                             const float* __restrict__ inv, float* __restrict__ X) {
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  // (a matrix of zeros stays one with eps = 0)
  const float s = isinf(*inv) ? 0.f : *inv;
  if (i < (long long)R * K) X[i] = to_f<T>(G[i / K * ld + i % K]) * s;
}

__global__ void k_orth_poly(const float* __restrict__ A, const float* __restrict__ A2, long long n,
                            float* __restrict__ P) {
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  if (i < n) P[i] = kB * A[i] + kC * A2[i];
}

__global__ void k_orth_axpy(const float* __restrict__ Y, long long n, float* __restrict__ X) {
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  if (i < n) X[i] = kA * X[i] + Y[i];
}

template <typename T>
__global__ void k_orth_out(const float* __restrict__ X, int R, int K, long long ld,
                           T* __restrict__ O) {
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  if (i < (long long)R * K) O[i / K * ld + i % K] = from_f<T>(X[i]);
}

struct OrthPlan {
  int R, K, N, m;
  long long ild, ib, old, ob;
  size_t w_inv, w_X, w_Y, w_A, w_A2, w_P, total;
};

bool orth_plan(const rnnt_orth_dims* d, OrthPlan* p) {
  if (!d || d->rows < 1 || d->cols < 1 || d->batch < 0 || d->steps < 1 || d->steps > 32)
    return false;
  if ((long long)d->rows * d->cols > 2147483647LL || !(d->eps >= 0.f)) return false;
  if (!op_dtype(d->in_dtype) || !op_dtype(d->out_dtype)) return false;
  p->R = d->rows; p->K = d->cols; p->N = d->batch;
  p->m = p->R < p->K ? p->R : p->K;
  p->ild = d->in_ld ? d->in_ld : p->K;
  p->ib = d->in_batch ? d->in_batch : p->R * p->ild;
  p->old = d->out_ld ? d->out_ld : p->K;
  p->ob = d->out_batch ? d->out_batch : p->R * p->old;
  if (p->ild < p->K || p->old < p->K) return false;
  if (p->N > 1 && (p->ib < 0 || p->ob < (long long)(p->R - 1) * p->old + p->K)) return false;
  const size_t x = 4 * (size_t)p->R * p->K, a = 4 * (size_t)p->m * p->m;
  size_t o = 0;
  auto put = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes); return at; };
  p->w_inv = put(4);
  p->w_X = put(x);
  p->w_Y = put(x);
  p->w_A = put(a);
  p->w_A2 = put(a);
  p->w_P = put(a);
  p->total = o;
  return true;
}

}  // namespace
}  // namespace rnnt

using namespace rnnt;

extern "C" {

size_t rnnt_orth_workspace_bytes(const rnnt_orth_dims* dims) {
  OrthPlan p;
  return orth_plan(dims, &p) ? p.total : 0;
}

rnnt_status rnnt_orth(const rnnt_orth_dims* dims, const void* G, void* O, void* ws,
                      size_t ws_bytes, int32_t* status, rnnt_stream stream) {
  OrthPlan p;
  if (!orth_plan(dims, &p)) return RNNT_ERR_INVALID_ARG;
  if (p.N == 0) return RNNT_OK;
  if (!G || !O || !ws) return RNNT_ERR_INVALID_ARG;
  if (!aligned_to(G, op_size(dims->in_dtype)) || !aligned_to(O, op_size(dims->out_dtype)) ||
      !aligned_to(ws, ALIGN) || !aligned_to(status, 4))
    return RNNT_ERR_INVALID_ARG;
  if (ws_bytes < p.total) return RNNT_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = (cudaStream_t)stream;
  char* w = (char*)ws;
  float *inv = (float*)(w + p.w_inv), *X = (float*)(w + p.w_X), *Y = (float*)(w + p.w_Y),
        *A = (float*)(w + p.w_A), *A2 = (float*)(w + p.w_A2), *P = (float*)(w + p.w_P);
  const long long n = (long long)p.R * p.K, mm = (long long)p.m * p.m;
  const int gx = (int)cdiv(n, 256), gm = (int)cdiv(mm, 256);
  const bool wide = p.R <= p.K;
  for (int i = 0; i < p.N; ++i) {
    const float* gf = (const float*)G + i * p.ib;
    const __nv_bfloat16* gb = (const __nv_bfloat16*)G + i * p.ib;
    if (dims->in_dtype == RNNT_F32) {
      k_orth_norm<<<1, 1024, 0, st>>>(gf, p.R, p.K, p.ild, dims->eps, inv);
      k_orth_scale<<<gx, 256, 0, st>>>(gf, p.R, p.K, p.ild, inv, X);
    } else {
      k_orth_norm<<<1, 1024, 0, st>>>(gb, p.R, p.K, p.ild, dims->eps, inv);
      k_orth_scale<<<gx, 256, 0, st>>>(gb, p.R, p.K, p.ild, inv, X);
    }
    OPS_CHECK(cudaGetLastError());
    for (int k = 0; k < dims->steps; ++k) {
      SimtGemm g{};
      g.alpha = 1.f;
      g.M = g.N = p.m; g.K = wide ? p.K : p.R;
      g.A = X; g.sam = wide ? p.K : 1; g.sak = wide ? 1 : p.K;
      g.Bm = X; g.sbn = g.sam; g.sbk = g.sak;
      g.C = A; g.ldc = p.m;
      OPS_LAUNCH("orth_gemm", launch_simt_gemm(g, st));
      g.K = p.m;
      g.A = A; g.sam = p.m; g.sak = 1;
      g.Bm = A; g.sbk = p.m; g.sbn = 1;
      g.C = A2;
      OPS_LAUNCH("orth_gemm", launch_simt_gemm(g, st));
      k_orth_poly<<<gm, 256, 0, st>>>(A, A2, mm, P);
      g.M = p.R; g.N = p.K;
      g.A = wide ? P : X; g.sam = wide ? p.m : p.K; g.sak = 1;
      g.Bm = wide ? X : P; g.sbk = wide ? p.K : p.m; g.sbn = 1;
      g.C = Y; g.ldc = p.K;
      OPS_LAUNCH("orth_gemm", launch_simt_gemm(g, st));
      k_orth_axpy<<<gx, 256, 0, st>>>(Y, n, X);
      OPS_CHECK(cudaGetLastError());
    }
    if (dims->out_dtype == RNNT_F32)
      k_orth_out<<<gx, 256, 0, st>>>(X, p.R, p.K, p.old, (float*)O + i * p.ob);
    else
      k_orth_out<<<gx, 256, 0, st>>>(X, p.R, p.K, p.old, (__nv_bfloat16*)O + i * p.ob);
    OPS_CHECK(cudaGetLastError());
  }
  return RNNT_OK;
}

}  // extern "C"
