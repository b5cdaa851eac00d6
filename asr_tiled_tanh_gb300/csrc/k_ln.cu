// k_ln.cu -- layer norm of rows, channels last (include/rnnt_ops.h).
#include <algorithm>

#include "ops.h"
#include "ptx.cuh"

namespace rnnt {
namespace {

struct LnArgs {
  int B, T, C, extra;  // extra: rows past lengths[b] that exist (1 for label rows)
  int rows;            // B * T
  float eps, rC;
  FastDiv t_div;
  long long xf, xb, yf, yb;
  const float* gamma;
  const float* beta;
  const int32_t* lengths;
  int32_t* status;
  float2* stats;  // mean and rstd of every row
};

// Row r of the batch.
struct Row {
  bool live;
  long long x, y;  // offsets of its first element
};
__device__ __forceinline__ Row row_of(const LnArgs& a, int r) {
  const int b = r / a.t_div, t = r - b * a.T;
  Row w;
  w.x = b * a.xb + t * a.xf;
  w.y = b * a.yb + t * a.yf;
  w.live = true;
  if (a.lengths) {
    const int n = __ldg(a.lengths + b);
    if (n < 0 || n > a.T - a.extra) {
      report(a.status, RNNT_ERR_LENGTH_RANGE);
      w.live = false;
    } else {
      w.live = t < n + a.extra;
    }
  }
  return w;
}

// ---- a block a row ------------------------------------------------------------
// Any width and alignment: the row is read again for each of its sums (from L2).
constexpr int WT = 256, WWARPS = WT / 32;

// Sums of two values over the block, for all threads; scr: 2 WWARPS + 2 floats.
__device__ __forceinline__ float2 block_sum(float2 v, float2* scr) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
  }
  __syncthreads();  // (scr may still be read)
  if ((threadIdx.x & 31) == 0) scr[threadIdx.x >> 5] = v;
  __syncthreads();
  v = scr[0];
#pragma unroll
  for (int k = 1; k < WWARPS; ++k) {
    v.x += scr[k].x;
    v.y += scr[k].y;
  }
  return v;
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(WT)
k_ln_fwd_wide(LnArgs a, const TX* __restrict__ x, TY* __restrict__ y) {
  __shared__ float2 scr[WWARPS];
  for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const Row w = row_of(a, r);
    TY* yr = y + w.y;
    if (!w.live) {
      for (int c = threadIdx.x; c < a.C; c += WT) yr[c] = from_f<TY>(0.f);
      continue;
    }
    const TX* xr = x + w.x;
    float2 s = make_float2(0.f, 0.f);
    for (int c = threadIdx.x; c < a.C; c += WT) s.x += to_f<TX>(xr[c]);
    const float mean = block_sum(s, scr).x / (float)a.C;  // (exact for rows of one value)
    s.x = 0.f;
    for (int c = threadIdx.x; c < a.C; c += WT) {
      const float d = to_f<TX>(xr[c]) - mean;
      s.x = fmaf(d, d, s.x);
    }
    const float rstd = 1.f / sqrtf(block_sum(s, scr).x * a.rC + a.eps);
    if (a.stats && threadIdx.x == 0) a.stats[r] = make_float2(mean, rstd);
    for (int c = threadIdx.x; c < a.C; c += WT) {
      const float xh = (to_f<TX>(xr[c]) - mean) * rstd;
      yr[c] = from_f<TY>(fmaf(a.gamma ? __ldg(a.gamma + c) : 1.f, xh,
                              a.beta ? __ldg(a.beta + c) : 0.f));
    }
  }
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(WT)
k_ln_bwd_wide(LnArgs a, const TX* __restrict__ x, const TY* __restrict__ dy,
              TX* __restrict__ dx) {
  __shared__ float2 scr[WWARPS];
  for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const Row w = row_of(a, r);
    TX* dr = dx + w.x;
    if (!w.live) {
      for (int c = threadIdx.x; c < a.C; c += WT) dr[c] = from_f<TX>(0.f);
      continue;
    }
    const TX* xr = x + w.x;
    const TY* gr = dy + w.y;
    const float2 st = a.stats[r];
    float2 s = make_float2(0.f, 0.f);
    for (int c = threadIdx.x; c < a.C; c += WT) {
      const float g = to_f<TY>(gr[c]) * (a.gamma ? __ldg(a.gamma + c) : 1.f);
      s.x += g;
      s.y = fmaf(g, (to_f<TX>(xr[c]) - st.x) * st.y, s.y);
    }
    s = block_sum(s, scr);
    const float m1 = s.x * a.rC, m2 = s.y * a.rC;
    for (int c = threadIdx.x; c < a.C; c += WT) {
      const float g = to_f<TY>(gr[c]) * (a.gamma ? __ldg(a.gamma + c) : 1.f);
      const float xh = (to_f<TX>(xr[c]) - st.x) * st.y;
      dr[c] = from_f<TX>(st.y * (g - m1 - xh * m2));
    }
  }
}

// part[slice][c] = (sum dy xh, sum dy) over the slice's rows: 32 channels and a
// slice of the rows a block.
template <typename TX, typename TY>
__global__ void __launch_bounds__(WT)
k_ln_cols(LnArgs a, const TX* __restrict__ x, const TY* __restrict__ dy,
          float2* __restrict__ part, int per) {
  __shared__ float2 scr[WWARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const long long r0 = (long long)blockIdx.y * per, r1 = min((long long)a.rows, r0 + per);
  float2 s = make_float2(0.f, 0.f);
  if (c < a.C)
    for (long long r = r0 + warp; r < r1; r += WWARPS) {
      const Row w = row_of(a, (int)r);
      if (!w.live) continue;
      const float2 st = a.stats[r];
      const float g = to_f<TY>(dy[w.y + c]);
      s.x = fmaf(g, (to_f<TX>(x[w.x + c]) - st.x) * st.y, s.x);
      s.y += g;
    }
  scr[warp][lane] = s;
  __syncthreads();
  if (warp || c >= a.C) return;
  for (int k = 1; k < WWARPS; ++k) {
    s.x += scr[k][lane].x;
    s.y += scr[k][lane].y;
  }
  part[(long long)blockIdx.y * a.C + c] = s;
}

// dgamma, dbeta: the column sums of part [n][C], 32 channels a block.
__global__ void __launch_bounds__(WT)
k_ln_params(const float2* __restrict__ part, int n, int C, float* __restrict__ dgamma,
            float* __restrict__ dbeta) {
  __shared__ float2 scr[WWARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float2 s = make_float2(0.f, 0.f);
  if (c < C)
#pragma unroll 4
    for (int r = warp; r < n; r += WWARPS) {
      const float2 p = __ldcg(part + (long long)r * C + c);
      s.x += p.x;
      s.y += p.y;
    }
  scr[warp][lane] = s;
  __syncthreads();
  if (warp || c >= C) return;
  for (int k = 1; k < WWARPS; ++k) {
    s.x += scr[k][lane].x;
    s.y += scr[k][lane].y;
  }
  if (dgamma) dgamma[c] = s.x;
  if (dbeta) dbeta[c] = s.y;
}

// Rows of `n` by strides: samples after one another, or frames after one another.
// (A tensor spans at most 2^47 elements, so that offsets stay within 64 bits.)
bool ln_strides(long long B, long long T, long long C, long long f, long long b) {
  const long long most = 1LL << 47;
  if (f < 0 || b < 0 || f > most || b > most) return false;
  if ((B > 1 && b > most / B) || (T > 1 && f > most / T)) return false;
  const bool by_sample = (T == 1 || f >= C) && (B <= 1 || b >= (T - 1) * f + C);
  const bool by_frame = (B <= 1 || b >= C) && (T == 1 || f >= (B - 1) * b + C);
  return by_sample || by_frame;
}

bool ln_args(const rnnt_ln_dims* d, LnArgs* a) {
  if (!d || d->B < 0 || d->T < 1 || d->C < 1) return false;
  if ((long long)d->B * d->T > (1LL << 30) || d->C > (1 << 20)) return false;
  if (!op_dtype(d->x_dtype) || !op_dtype(d->y_dtype) || !(d->eps >= 0.f)) return false;
  a->B = d->B; a->T = d->T; a->C = d->C; a->extra = d->label_rows != 0;
  a->rows = d->B * d->T;
  a->eps = d->eps;
  a->rC = 1.f / (float)d->C;
  a->t_div = fast_div(d->T);
  const long long most = 1LL << 47;  // (before a product of strides is taken)
  if (d->x_frame < 0 || d->x_frame > most || d->y_frame < 0 || d->y_frame > most) return false;
  a->xf = d->x_frame ? d->x_frame : d->C;
  a->yf = d->y_frame ? d->y_frame : d->C;
  if (a->xf > most / d->T || a->yf > most / d->T) return false;
  a->xb = d->x_batch ? d->x_batch : d->T * a->xf;
  a->yb = d->y_batch ? d->y_batch : d->T * a->yf;
  return ln_strides(d->B, d->T, d->C, a->xf, a->xb) && ln_strides(d->B, d->T, d->C, a->yf, a->yb);
}

// Slices of the rows whose sums the workspace holds.
int ln_slices(const LnArgs& a) {
  return (int)std::min<long long>(64, std::max(1, a.rows));
}

rnnt_status ln_check(const rnnt_ln_dims* d, LnArgs* a, const void* x, const void* y,
                     const float* gamma, const float* beta, const int32_t* lengths,
                     const void* saved, int32_t* status) {
  if (!ln_args(d, a)) return RNNT_ERR_INVALID_ARG;
  if (a->rows > 0 && (!x || !y)) return RNNT_ERR_INVALID_ARG;
  if (!aligned_to(x, op_size(d->x_dtype)) || !aligned_to(y, op_size(d->y_dtype)) ||
      !aligned_to(gamma, 4) || !aligned_to(beta, 4) || !aligned_to(lengths, 4) ||
      !aligned_to(saved, ALIGN) || !aligned_to(status, 4))
    return RNNT_ERR_INVALID_ARG;
  a->gamma = gamma; a->beta = beta; a->lengths = lengths; a->status = status;
  a->stats = (float2*)saved;
  return RNNT_OK;
}

template <typename TX, typename TY>
cudaError_t ln_fwd(const LnArgs& a, const void* x, void* y, cudaStream_t st) {
  const int grid = std::min(a.rows, 8 * num_sms());
  k_ln_fwd_wide<TX, TY><<<grid, WT, 0, st>>>(a, (const TX*)x, (TY*)y);
  return cudaGetLastError();
}

template <typename TX, typename TY>
cudaError_t ln_bwd(const LnArgs& a, const void* x, const void* dy, void* dx, float2* part,
                   bool params, cudaStream_t st) {
  const int grid = std::min(a.rows, 8 * num_sms());
  k_ln_bwd_wide<TX, TY><<<grid, WT, 0, st>>>(a, (const TX*)x, (const TY*)dy, (TX*)dx);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !params) return e;
  const int n = ln_slices(a);
  k_ln_cols<TX, TY><<<dim3((unsigned)cdiv(a.C, 32), n), WT, 0, st>>>(
      a, (const TX*)x, (const TY*)dy, part, (int)cdiv(a.rows, n));
  return cudaGetLastError();
}

}  // namespace
}  // namespace rnnt

using namespace rnnt;

extern "C" {

size_t rnnt_ln_saved_bytes(const rnnt_ln_dims* dims) {
  LnArgs a;
  return ln_args(dims, &a) ? align_up(8 * (size_t)a.rows + 8) : 0;
}

size_t rnnt_ln_workspace_bytes(const rnnt_ln_dims* dims) {
  LnArgs a;
  return ln_args(dims, &a) ? align_up(8 * (size_t)ln_slices(a) * a.C) : 0;
}

rnnt_status rnnt_ln_fwd(const rnnt_ln_dims* dims, const void* x, const float* gamma,
                        const float* beta, const int32_t* lengths, void* y, void* saved,
                        int32_t* status, rnnt_stream stream) {
  LnArgs a;
  const rnnt_status s = ln_check(dims, &a, x, y, gamma, beta, lengths, saved, status);
  if (s != RNNT_OK) return s;
  if (a.rows == 0) return RNNT_OK;
  cudaStream_t st = (cudaStream_t)stream;
  using bf = __nv_bfloat16;
  const bool yf = dims->y_dtype == RNNT_F32;
  if (dims->x_dtype == RNNT_F32)
    OPS_LAUNCH("ln_fwd", (yf ? ln_fwd<float, float>(a, x, y, st) : ln_fwd<float, bf>(a, x, y, st)));
  else
    OPS_LAUNCH("ln_fwd", (yf ? ln_fwd<bf, float>(a, x, y, st) : ln_fwd<bf, bf>(a, x, y, st)));
  return RNNT_OK;
}

rnnt_status rnnt_ln_bwd(const rnnt_ln_dims* dims, const void* x, const void* dy,
                        const float* gamma, const int32_t* lengths, const void* saved, void* dx,
                        float* dgamma, float* dbeta, void* ws, size_t ws_bytes, int32_t* status,
                        rnnt_stream stream) {
  LnArgs a;
  const rnnt_status s = ln_check(dims, &a, x, dy, gamma, nullptr, lengths, saved, status);
  if (s != RNNT_OK) return s;
  if ((a.rows > 0 && (!dx || !saved)) || !ws) return RNNT_ERR_INVALID_ARG;
  if (!aligned_to(dx, op_size(dims->x_dtype)) || !aligned_to(dgamma, 4) ||
      !aligned_to(dbeta, 4) || !aligned_to(ws, ALIGN))
    return RNNT_ERR_INVALID_ARG;
  if (ws_bytes < rnnt_ln_workspace_bytes(dims)) return RNNT_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = (cudaStream_t)stream;
  using bf = __nv_bfloat16;
  const bool yf = dims->y_dtype == RNNT_F32, params = dgamma || dbeta;
  float2* part = (float2*)ws;
  if (a.rows > 0) {
    ProfScope ps("ln_bwd", st);
    if (dims->x_dtype == RNNT_F32)
      OPS_CHECK((yf ? ln_bwd<float, float>(a, x, dy, dx, part, params, st)
                    : ln_bwd<float, bf>(a, x, dy, dx, part, params, st)));
    else
      OPS_CHECK((yf ? ln_bwd<bf, float>(a, x, dy, dx, part, params, st)
                    : ln_bwd<bf, bf>(a, x, dy, dx, part, params, st)));
  }
  if (!params) return RNNT_OK;
  ProfScope ps("ln_params", st);
  k_ln_params<<<(unsigned)cdiv(a.C, 32), WT, 0, st>>>(part, a.rows ? ln_slices(a) : 0, a.C, dgamma,
                                                     dbeta);
  OPS_CHECK(cudaGetLastError());
  return RNNT_OK;
}

}  // extern "C"
