// k_ln_bwd.cu -- layer norm of rows: the backward pass (include/rnnt_ops.h).
#include "ln.cuh"

namespace rnnt {
namespace {
using namespace ln;

// dx of the team's rows, and part[block][c] = (sum dy xh, sum dy) over the block's.
template <typename TX, typename TY, int VEC, int NV>
__global__ void __launch_bounds__(MAX_THREADS)
k_ln_bwd(LnArgs a, Team t, const TX* __restrict__ x, const TY* __restrict__ dy,
         TX* __restrict__ dx, float2* __restrict__ part) {
  using RX = Ring<VEC, NV, TX>;
  using RY = Ring<VEC, NV, TY>;
  constexpr int NP = kPairs(VEC);
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float scr[2][MAX_THREADS / 32][2];
  const Place p = place_of(t);
  const bool al16 = ((uintptr_t)a.gamma & 15) == 0;
  RX rx;
  RY ry;
  rx.init(smem);
  ry.init(smem + RX::bytes(blockDim.x));
  unsigned lives = 0;
  int length = ask_length(a, p.first);
  auto ahead = [&](int r, int stage) {
    const bool live = exists(a, r, length, p.lane == 0);
    length = ask_length(a, r + p.step);
    if (live) {
      rx.fetch(stage, x + offset(r, a, a.xf, a.xb), t, p);
      ry.fetch(stage, dy + offset(r, a, a.yf, a.yb), t, p);
    }
    copy_commit();
    lives = (lives & ~(1u << stage)) | ((unsigned)live << stage);
  };
#pragma unroll
  for (int s = 0; s < STAGES; ++s) ahead(p.first + s * p.step, s);
  auto ask_stats = [&](int r, bool live) {
    return live ? __ldg(a.stats + r) : make_float2(0.f, 0.f);
  };
  float2 next = ask_stats(p.first, lives & 1);
  Vals<VEC> gamma[NV], dg[NV], db[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int k = p.lane + j * t.lanes;
    if (k < t.nvec) gamma[j] = param<VEC>(a.gamma, k * VEC, 1.f, al16);
    else gamma[j].fill(0.f);
    dg[j].fill(0.f);
    db[j].fill(0.f);
  }
  int stage = 0, par = 0;
#pragma unroll 1
  for (int r = p.first, w = p.warp0; w < a.rows; r += p.step, w += p.step) {
    const bool live = (lives >> stage) & 1;
    const long long at = offset(r, a, a.xf, a.xb);
    TX* dr = dx + at;
    typename RX::U ux[NV];
    typename RY::U uy[NV];
    copy_wait<STAGES - 1>();
    rx.read(ux, stage, x + (RX::kAhead ? 0 : at), live, t, p);
    ry.read(uy, stage, dy + (RY::kAhead ? 0 : offset(r, a, a.yf, a.yb)), live, t, p);
    ahead(r + STAGES * p.step, stage);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    const float2 st = next;
    next = ask_stats(r + p.step, (lives >> stage) & 1);
    if (t.lanes < 32 ? !__any_sync(0xffffffffu, live) : !live) {
      Vals<VEC> z;
      z.fill(0.f);
      if (r < a.rows)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int k = p.lane + j * t.lanes;
          if (k < t.nvec) store<VEC, TX>(dr + k * VEC, z);
        }
      continue;
    }
    // (rows and vectors that do not exist: dy is 0)
    Vals<VEC> xh[NV], g[NV];
    float2 s1 = make_float2(0.f, 0.f), s2 = s1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xh[j] = widen<VEC, TX>(ux[j]);
      g[j] = widen<VEC, TY>(uy[j]);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        xh[j].p[i] = __fmul2_rn(__fadd2_rn(xh[j].p[i], make_float2(-st.x, -st.x)),
                                make_float2(st.y, st.y));
        dg[j].p[i] = __ffma2_rn(g[j].p[i], xh[j].p[i], dg[j].p[i]);
        db[j].p[i] = __fadd2_rn(g[j].p[i], db[j].p[i]);
        g[j].p[i] = __fmul2_rn(g[j].p[i], gamma[j].p[i]);
        s1 = __fadd2_rn(g[j].p[i], s1);
        s2 = __ffma2_rn(g[j].p[i], xh[j].p[i], s2);
      }
    }
    float s[2] = {s1.x + s1.y, s2.x + s2.y};
    team_sum(s, t, p, scr[par]);
    par ^= 1;
    const float m1 = -s[0] * a.rC, m2 = -s[1] * a.rC;
    if (r < a.rows)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int k = p.lane + j * t.lanes;
        if (k >= t.nvec) continue;
        Vals<VEC> o;
#pragma unroll
        for (int i = 0; i < NP; ++i)
          o.p[i] = __fmul2_rn(__ffma2_rn(xh[j].p[i], make_float2(m2, m2),
                                         __fadd2_rn(g[j].p[i], make_float2(m1, m1))),
                              make_float2(st.y, st.y));
        store<VEC, TX>(dr + k * VEC, o);
      }
  }
  copy_wait<0>();
  if (!part) return;
  // the block's sums: the teams' in order (of a warp's narrow teams by shuffles first)
  const int groups = t.lanes < 32 ? (int)blockDim.x >> 5 : t.teams;
  const int cols = t.lanes * VEC, group = t.lanes < 32 ? (int)threadIdx.x >> 5 : p.team;
  float2* sums = (float2*)smem;  // [group][cols]
  float2* row = part + (long long)blockIdx.x * a.C;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float2 v = make_float2(i & 1 ? dg[j].p[i / 2].y : dg[j].p[i / 2].x,
                             i & 1 ? db[j].p[i / 2].y : db[j].p[i / 2].x);
      for (int d = 16; d >= t.lanes; d >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
      }
      // (lanes next to each other, so that their stores do not meet in a bank)
      sums[group * cols + i * t.lanes + p.lane] = v;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
      const int lane = c / VEC, at = (c - lane * VEC) * t.lanes + lane;
      const int col = j * cols + c;
      if (col >= a.C) continue;
      float2 v = sums[at];
      for (int k = 1; k < groups; ++k) v = __fadd2_rn(v, sums[k * cols + at]);
      row[col] = v;
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

constexpr int PART_ROWS = 608;  // (the workspace may not depend on the device)

template <typename TX, typename TY, int VEC, int NV>
cudaError_t bwd_team(const LnArgs& a, const Team& t, const void* x, const void* dy, void* dx,
                     float2* part, int* part_rows, cudaStream_t st) {
  static Known known;
  const int threads = t.lanes * t.teams;
  const size_t sums = sizeof(float2) * VEC * threads;
  const size_t smem =
      std::max(sums, Ring<VEC, NV, TX>::bytes(threads) + Ring<VEC, NV, TY>::bytes(threads));
  int per = 0;
  const cudaError_t e = blocks_per_sm(k_ln_bwd<TX, TY, VEC, NV>, &known, threads, smem, &per);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<long long>(
      std::min<long long>(cdiv(a.rows, t.teams), part_rows_max(a)), (long long)per * num_sms());
  k_ln_bwd<TX, TY, VEC, NV><<<grid, threads, smem, st>>>(a, t, (const TX*)x, (const TY*)dy, (TX*)dx,
                                                         part);
  *part_rows = grid;
  return cudaGetLastError();
}

template <typename TX, typename TY>
cudaError_t ln_bwd(const LnArgs& a, const void* x, const void* dy, void* dx, float2* part,
                   int* part_rows, cudaStream_t st) {
  constexpr int V16 = 16 / (int)std::max(sizeof(TX), sizeof(TY));
  const int vec = vec_of(a, sizeof(TX), x, dx, sizeof(TY), dy);
  int nv = 0;
  // (16 channels a lane: their sums stay in registers)
  const Team t = team_for((int)cdiv(a.C, vec), vec == V16 ? 16 / V16 : 8, vec == V16, &nv);
  if (t.lanes) {
    if (vec == V16) switch (nv) {
      case 1: return bwd_team<TX, TY, V16, 1>(a, t, x, dy, dx, part, part_rows, st);
      case 2: return bwd_team<TX, TY, V16, 2>(a, t, x, dy, dx, part, part_rows, st);
      default:
        if constexpr (V16 == 4) {
          if (nv == 3) return bwd_team<TX, TY, V16, 3>(a, t, x, dy, dx, part, part_rows, st);
          return bwd_team<TX, TY, V16, 4>(a, t, x, dy, dx, part, part_rows, st);
        }
    }
    if (vec == 2) switch (nv) {
      case 2: return bwd_team<TX, TY, 2, 2>(a, t, x, dy, dx, part, part_rows, st);
      case 4: return bwd_team<TX, TY, 2, 4>(a, t, x, dy, dx, part, part_rows, st);
      default: return bwd_team<TX, TY, 2, 8>(a, t, x, dy, dx, part, part_rows, st);
    }
    switch (nv) {
      case 2: return bwd_team<TX, TY, 1, 2>(a, t, x, dy, dx, part, part_rows, st);
      case 4: return bwd_team<TX, TY, 1, 4>(a, t, x, dy, dx, part, part_rows, st);
      default: return bwd_team<TX, TY, 1, 8>(a, t, x, dy, dx, part, part_rows, st);
    }
  }
  const int grid = std::min(a.rows, 8 * num_sms());
  k_ln_bwd_wide<TX, TY><<<grid, WT, 0, st>>>(a, (const TX*)x, (const TY*)dy, (TX*)dx);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !part) return e;
  const int n = std::min(64, part_rows_max(a));
  k_ln_cols<TX, TY><<<dim3((unsigned)cdiv(a.C, 32), n), WT, 0, st>>>(
      a, (const TX*)x, (const TY*)dy, part, (int)cdiv(a.rows, n));
  *part_rows = n;
  return cudaGetLastError();
}

}  // namespace

namespace ln {

int part_rows_max(const LnArgs& a) { return std::min(PART_ROWS, std::max(1, a.rows)); }

cudaError_t launch_bwd(const LnArgs& a, int x_dtype, int y_dtype, const void* x, const void* dy,
                       void* dx, float2* part, int* part_rows, bool params, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (!params) part = nullptr;
  if (x_dtype == RNNT_F32)
    return y_dtype == RNNT_F32 ? ln_bwd<float, float>(a, x, dy, dx, part, part_rows, st)
                               : ln_bwd<float, bf>(a, x, dy, dx, part, part_rows, st);
  return y_dtype == RNNT_F32 ? ln_bwd<bf, float>(a, x, dy, dx, part, part_rows, st)
                             : ln_bwd<bf, bf>(a, x, dy, dx, part, part_rows, st);
}

cudaError_t launch_params(const float2* part, int rows, int C, float* dgamma, float* dbeta,
                          cudaStream_t st) {
  k_ln_params<<<(unsigned)cdiv(C, 32), WT, 0, st>>>(part, rows, C, dgamma, dbeta);
  return cudaGetLastError();
}

}  // namespace ln
}  // namespace rnnt
