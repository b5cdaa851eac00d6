// k_ln.cu -- layer norm of rows, channels last (include/rnnt_ops.h): the forward
// pass, and the checks of both.
#include "ln.cuh"

namespace rnnt {
namespace {
using namespace ln;

// Rows ahead.  What is read ahead competes with what is written (us with one, two and
// three stages): 1024 x 1000 x 256 and 64 x 1000 x 4096, all fp32, 321, 344, 341 and 328,
// 347, 361; fp32 to bf16 260, 250, 263 and 261, 227, 244; bf16 to fp32 274, 242, 264 and
// 273, 253, 254; bf16 in two units a lane, 512 x 1000 x 1024, 387, 332, 324; in three,
// 512 x 1000 x 640, 704 and 768, 231, 199, 198 and 248, 233, 250 and 258, 268, 275; parts
// of a warp, 512 x 2000 x 64 in fp32, 97, 85, 85.
template <typename TX, typename TY, int VEC, int NV, int MODE>
constexpr int stages() {
  if (!kCopied<VEC, TX>) return 1;
  if (sizeof(TX) != sizeof(TY) || (VEC == 8 && NV == 3)) return 2;
  return sizeof(TX) == 4 && VEC == 4 && MODE != PART ? 1 : STAGES;
}

template <typename TX, typename TY, int VEC, int NV, int MODE>
__global__ void
__launch_bounds__(MODE == WARPS ? MAX_THREADS : 256, MODE == WARPS ? 1 : 2)
k_ln_fwd(LnArgs a, Team t, const TX* __restrict__ x, TY* __restrict__ y) {
  constexpr int NP = kPairs(VEC), S = stages<TX, TY, VEC, NV, MODE>();
  using R = Ring<VEC, NV, S, TX>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float scr[2][MAX_THREADS / 32][1];
  const Place p = place_of<MODE>(t);
  const bool al16 = (((uintptr_t)a.gamma | (uintptr_t)a.beta) & 15) == 0;
  const Cols<VEC> cols{p.lane, t.lanes, a.C};
  const Stride by(a, p.step);
  // the row to copy next, and the row at hand
  Walk next(a, p.first), row = next;
  Offset xo(a, next, by, a.xf, a.xb), yo(a, row, by, a.yf, a.yb);
  R ring;
  ring.init(smem);
  __syncthreads();
  unsigned lives = 0;  // bit s: the row s turns from now exists
  int length = ask_length(a, next);
  auto ahead = [&](int stage) {
    const bool live = exists(a, next, length, p.lane == 0);
    if (live) ring.fetch(stage, x + xo.at, cols);
    copy_commit();
    lives |= (unsigned)live << (S - 1);
    advance(a, by, next, xo);
    length = ask_length(a, next);
  };
#pragma unroll
  for (int s = 0; s < S; ++s) {
    lives >>= 1;
    ahead(s);
  }
  Vals<VEC> gamma[NV], beta[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    gamma[j] = cols.param(a.gamma, j, 1.f, al16);
    beta[j] = cols.param(a.beta, j, 0.f, al16);
  }
  const float C = (float)a.C;
  int stage = 0;
#pragma unroll 1
  while (MODE == PART ? __any_sync(0xffffffffu, row.b < a.B) : row.b < a.B) {
    const bool live = lives & 1, here = MODE != PART || row.b < a.B;
    const int r = row.b * a.T + row.t;
    TY* to = y + yo.at;
    typename R::U u[NV];
    copy_wait<S - 1>();
    ring.read(u, stage);
    lives >>= 1;
    ahead(stage);
    stage = stage + 1 == S ? 0 : stage + 1;
    advance(a, by, row, yo);
    if (MODE == PART ? !__any_sync(0xffffffffu, live) : !live) {
      Vals<VEC> z;
      z.fill(0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (here) cols.store(to, j, z);
      continue;
    }
    // the mean, then the squares about it
    Vals<VEC> v[NV];
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      v[j] = widen<VEC, TX>(u[j]);
#pragma unroll
      for (int i = 0; i < NP; ++i) s2 = __fadd2_rn(s2, v[j].p[i]);
    }
    float s[1] = {s2.x + s2.y};
    team_sum<MODE>(s, t, p, scr[0]);
    float mean = s[0] * a.rC;
    mean = fmaf(fmaf(-mean, C, s[0]), a.rC, mean);  // (the sum's quotient, rounded once)
    s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        v[j].p[i] = __fadd2_rn(v[j].p[i], make_float2(-mean, -mean));
        if (VEC == 1 && !cols.both(j)) v[j].p[i].y = 0.f;
        if (cols.has(j)) s2 = __ffma2_rn(v[j].p[i], v[j].p[i], s2);
      }
    }
    s[0] = s2.x + s2.y;
    team_sum<MODE>(s, t, p, scr[1]);
    // (what a sum of equal bf16 values needs, 8 bits and those of C, it has)
    const bool flat = sizeof(TX) == 4 && may_be_flat(s[0], a.rC, mean);
    if (MODE == PART ? sizeof(TX) == 4 && __any_sync(0xffffffffu, flat) : flat) {
      // (a warp's other teams only keep the flat ones company: by 0)
      s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (cols.has(j)) s2 = __fadd2_rn(s2, v[j].p[i]);
      float rest[1] = {s2.x + s2.y};
      team_sum<MODE>(rest, t, p, scr[0]);
      const float better = flat ? fmaf(rest[0], a.rC, mean) : mean, off = better - mean;
      mean = better;
      s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          v[j].p[i] = __fadd2_rn(v[j].p[i], make_float2(-off, -off));
          if (VEC == 1 && !cols.both(j)) v[j].p[i].y = 0.f;
          if (cols.has(j)) s2 = __ffma2_rn(v[j].p[i], v[j].p[i], s2);
        }
      }
      s[0] = s2.x + s2.y;
      team_sum<MODE>(s, t, p, scr[1]);
    }
    const float rstd = root_of(fmaf(s[0], a.rC, a.eps));
    if (a.stats && live && p.lane == 0) a.stats[r] = make_float2(mean, rstd);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Vals<VEC> o;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        o.p[i] = __ffma2_rn(gamma[j].p[i], __fmul2_rn(v[j].p[i], make_float2(rstd, rstd)),
                            beta[j].p[i]);
        if (MODE == PART && !live) o.p[i] = make_float2(0.f, 0.f);
      }
      if (here) cols.store(to, j, o);
    }
  }
  copy_wait<0>();
}

template <typename TX, typename TY, int VEC>
__global__ void __launch_bounds__(WT)
k_ln_fwd_wide(LnArgs a, const TX* __restrict__ x, TY* __restrict__ y) {
  constexpr int NP = kPairs(VEC);
  __shared__ float2 scr[WWARPS];
  const Cols<VEC> cols{(int)threadIdx.x, WT, a.C};
  const bool al16 = (((uintptr_t)a.gamma | (uintptr_t)a.beta) & 15) == 0;
  for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const Row w = row_of(a, r);
    TY* yr = y + w.y;
    if (!w.live) {
      Vals<VEC> z;
      z.fill(0.f);
      for (int j = 0; cols.has(j); ++j) cols.store(yr, j, z);
      continue;
    }
    const TX* xr = x + w.x;
    float2 s = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int j = 0; cols.has(j); ++j) {
      const Vals<VEC> v = cols.load(xr, j);
#pragma unroll
      for (int i = 0; i < NP; ++i) s = __fadd2_rn(s, v.p[i]);
    }
    float mean = block_sum(make_float2(s.x + s.y, 0.f), scr).x / (float)a.C;
    // sums about the mean: of the squares, or of what is left
    auto about = [&](bool squares) {
      float2 q = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int j = 0; cols.has(j); ++j) {
        const Vals<VEC> v = cols.load(xr, j);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          float2 d = __fadd2_rn(v.p[i], make_float2(-mean, -mean));
          if (VEC == 1 && !cols.both(j)) d.y = 0.f;
          q = __ffma2_rn(d, squares ? d : make_float2(1.f, 1.f), q);
        }
      }
      return block_sum(make_float2(q.x + q.y, 0.f), scr).x;
    };
    float var = about(true);
    if (may_be_flat(var, a.rC, mean)) {
      mean = fmaf(about(false), a.rC, mean);
      var = about(true);
    }
    const float rstd = root_of(fmaf(var, a.rC, a.eps));
    if (a.stats && threadIdx.x == 0) a.stats[r] = make_float2(mean, rstd);
#pragma unroll 2
    for (int j = 0; cols.has(j); ++j) {
      const Vals<VEC> v = cols.load(xr, j), g = cols.param(a.gamma, j, 1.f, al16);
      Vals<VEC> o = cols.param(a.beta, j, 0.f, al16);
#pragma unroll
      for (int i = 0; i < NP; ++i)
        o.p[i] = __ffma2_rn(g.p[i], __fmul2_rn(__fadd2_rn(v.p[i], make_float2(-mean, -mean)),
                                               make_float2(rstd, rstd)), o.p[i]);
      cols.store(yr, j, o);
    }
  }
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
struct Fwd {
  const LnArgs& a;
  const void* x;
  void* y;
  cudaStream_t st;
  template <int VEC, int NV, int MODE>
  cudaError_t run(const Team& t) const {
    static Known known;
    const auto k = k_ln_fwd<TX, TY, VEC, NV, MODE>;
    const int threads = t.lanes * t.teams;
    const size_t smem = Ring<VEC, NV, stages<TX, TY, VEC, NV, MODE>(), TX>::bytes(threads);
    int per = 0;
    const cudaError_t e = blocks_per_sm(k, &known, threads, smem, &per);
    if (e != cudaSuccess) return e;
    const int grid = (int)std::min<long long>(cdiv(a.rows, t.teams), (long long)per * num_sms());
    k<<<grid, threads, smem, st>>>(a, t, (const TX*)x, (TY*)y);
    return cudaGetLastError();
  }
};

template <typename TX, typename TY>
cudaError_t ln_fwd(const LnArgs& a, const void* x, void* y, cudaStream_t st) {
  constexpr int V16 = 16 / (int)std::max(sizeof(TX), sizeof(TY));
  const int vec = vec_of(a, sizeof(TX), x, nullptr, sizeof(TY), y);
  cudaError_t e;
  const Fwd<TX, TY> f{a, x, y, st};
  if (by_team<V16, 24, 24, (V16 == 8 ? 24 : 16), 8>(a.C, vec, f, &e)) return e;
  const auto k = vec == V16 ? k_ln_fwd_wide<TX, TY, V16> : k_ln_fwd_wide<TX, TY, 1>;
  k<<<std::min(a.rows, 4 * num_sms()), WT, 0, st>>>(a, (const TX*)x, (TY*)y);
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
  return ln_args(dims, &a) ? align_up(8 * (size_t)part_rows_max(a) * a.C) : 0;
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
  const bool params = dgamma || dbeta;
  int rows = 0;
  if (a.rows > 0)
    OPS_LAUNCH("ln_bwd", launch_bwd(a, dims->x_dtype, dims->y_dtype, x, dy, dx, (float2*)ws, &rows,
                                    params, st));
  if (params)
    OPS_LAUNCH("ln_params", launch_params((const float2*)ws, rows, a.C, dgamma, dbeta, st));
  return RNNT_OK;
}

}  // extern "C"
