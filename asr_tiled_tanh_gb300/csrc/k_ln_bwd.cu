// k_ln_bwd.cu -- layer norm of rows: the backward pass (include/rnnt_ops.h).
#include "ln.cuh"

namespace rnnt {
namespace {
using namespace ln;

// Threads of a block at most.  Up to 16 channels a lane fit in 128 registers, two blocks
// of 256 threads an SM; 24 take 168, and three blocks of 128 (512 x 1000 rows of 640 in
// bf16: 322 us; with one block of 256 377, by two warps a row of 16 channels a lane 427).
template <int VEC, int NV, int MODE>
constexpr int kBound = VEC >= 4 && VEC * NV > 16 ? 128 : MODE == WARPS ? MAX_THREADS : 256;

// dx of the team's rows, and part[block][c] = (sum dy xh, sum dy) over the block's.
template <typename TX, typename TY, int VEC, int NV, int MODE>
__global__ void
__launch_bounds__(kBound<VEC, NV, MODE>,
                  kBound<VEC, NV, MODE> == 128 ? 3 : MODE == WARPS ? 1 : 2)
k_ln_bwd(LnArgs a, Team t, const TX* __restrict__ x, const TY* __restrict__ dy,
         TX* __restrict__ dx, float2* __restrict__ part) {
  constexpr int NP = kPairs(VEC), S = kCopied<VEC, TX> && kCopied<VEC, TY> ? STAGES : 1;
  using RX = Ring<VEC, NV, S, TX>;
  using RY = Ring<VEC, NV, S, TY>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float scr[2][MAX_THREADS / 32][2];
  ptx::griddep_launch();
  const Place p = place_of<MODE>(t);
  const bool al16 = ((uintptr_t)a.gamma & 15) == 0;
  const Cols<VEC> cols{p.lane, t.lanes, a.C};
  const Stride by(a, p.step);
  Walk next(a, p.first), row = next;
  Offset xo(a, next, by, a.xf, a.xb), yo(a, next, by, a.yf, a.yb), xr = xo;
  RX rx;
  RY ry;
  rx.init(smem);
  ry.init(smem + RX::bytes(blockDim.x));
  __syncthreads();
  unsigned lives = 0;  // bit s: the row s turns from now exists
  int length = ask_length(a, next);
  auto ahead = [&](int stage) {
    const bool live = exists(a, next, length, p.lane == 0);
    if (live) {
      rx.fetch(stage, x + xo.at, cols);
      ry.fetch(stage, dy + yo.at, cols);
    }
    copy_commit();
    lives |= (unsigned)live << (S - 1);
    advance(a, by, next, xo, yo);
    length = ask_length(a, next);
  };
#pragma unroll
  for (int s = 0; s < S; ++s) {
    lives >>= 1;
    ahead(s);
  }
  auto ask_stats = [&]() {
    return lives & 1 ? __ldg(a.stats + row.b * a.T + row.t) : make_float2(0.f, 0.f);
  };
  float2 coming = ask_stats();
  Vals<VEC> gamma[NV], dg[NV], db[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    gamma[j] = cols.param(a.gamma, j, 1.f, al16);
    dg[j].fill(0.f);
    db[j].fill(0.f);
  }
  int stage = 0, par = 0;
#pragma unroll 1
  while (MODE == PART ? __any_sync(0xffffffffu, row.b < a.B) : row.b < a.B) {
    const bool live = lives & 1, here = MODE != PART || row.b < a.B;
    TX* to = dx + xr.at;
    typename RX::U ux[NV];
    typename RY::U uy[NV];
    copy_wait<S - 1>();
    rx.read(ux, stage);
    ry.read(uy, stage);
    lives >>= 1;
    ahead(stage);
    stage = stage + 1 == S ? 0 : stage + 1;
    advance(a, by, row, xr);
    const float2 st = coming;
    coming = ask_stats();
    if (MODE == PART ? !__any_sync(0xffffffffu, live) : !live) {
      Vals<VEC> z;
      z.fill(0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (here) cols.store(to, j, z);
      continue;
    }
    // (of vectors past the row's end dy is 0)
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
        if (MODE == PART && !live) xh[j].p[i] = g[j].p[i] = make_float2(0.f, 0.f);
        dg[j].p[i] = __ffma2_rn(g[j].p[i], xh[j].p[i], dg[j].p[i]);
        db[j].p[i] = __fadd2_rn(g[j].p[i], db[j].p[i]);
        g[j].p[i] = __fmul2_rn(g[j].p[i], gamma[j].p[i]);
        s1 = __fadd2_rn(g[j].p[i], s1);
        s2 = __ffma2_rn(g[j].p[i], xh[j].p[i], s2);
      }
    }
    float s[2] = {s1.x + s1.y, s2.x + s2.y};
    team_sum<MODE>(s, t, p, scr[par]);
    par ^= 1;
    // dx = rstd a + (k1 + k2 xh)
    const float k1 = -s[0] * a.rC * st.y, k2 = -s[1] * a.rC * st.y;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Vals<VEC> o;
#pragma unroll
      for (int i = 0; i < NP; ++i)
        o.p[i] = __ffma2_rn(g[j].p[i], make_float2(st.y, st.y),
                            __ffma2_rn(xh[j].p[i], make_float2(k2, k2), make_float2(k1, k1)));
      if (here) cols.store(to, j, o);
    }
  }
  copy_wait<0>();
  if (!part) return;
  // the block's sums: the teams' in order (of a warp's narrow teams by shuffles first)
  constexpr int CH = 2 * NP;  // channels of a unit
  const int groups = MODE == WARPS ? t.teams : (int)blockDim.x >> 5;
  const int n = t.lanes * CH, group = MODE == WARPS ? p.team : (int)threadIdx.x >> 5;
  float2* sums = (float2*)smem;  // [group][channel of the lanes' units][lane]
  float2* out = part + (long long)blockIdx.x * a.C;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float2 v = make_float2(i & 1 ? dg[j].p[i / 2].y : dg[j].p[i / 2].x,
                             i & 1 ? db[j].p[i / 2].y : db[j].p[i / 2].x);
      for (int d = 16; MODE == PART && d >= t.lanes; d >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
      }
      sums[group * n + i * t.lanes + p.lane] = v;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      // (channels that are apart lie here as in the row)
      const int lane = VEC == 1 ? 0 : c / CH, at = VEC == 1 ? c : (c - lane * CH) * t.lanes + lane;
      if (j * n + c >= a.C) continue;
      float2 v = sums[at];
      for (int k = 1; k < groups; ++k) v = __fadd2_rn(v, sums[k * n + at]);
      out[j * n + c] = v;
    }
  }
}

template <typename TX, typename TY, int VEC>
__global__ void __launch_bounds__(WT)
k_ln_bwd_wide(LnArgs a, const TX* __restrict__ x, const TY* __restrict__ dy,
              TX* __restrict__ dx) {
  constexpr int NP = kPairs(VEC);
  __shared__ float2 scr[WWARPS];
  const Cols<VEC> cols{(int)threadIdx.x, WT, a.C};
  const bool al16 = ((uintptr_t)a.gamma & 15) == 0;
  for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const Row w = row_of(a, r);
    TX* dr = dx + w.x;
    if (!w.live) {
      Vals<VEC> z;
      z.fill(0.f);
      for (int j = 0; cols.has(j); ++j) cols.store(dr, j, z);
      continue;
    }
    const float2 st = a.stats[r];
    const TX* xr = x + w.x;
    const TY* gr = dy + w.y;
    // gamma dy and xh of unit j (past the row's end gamma is 0)
    auto terms = [&](int j, Vals<VEC>& g, Vals<VEC>& xh) {
      g = cols.load(gr, j);
      xh = cols.load(xr, j);
      const Vals<VEC> gamma = cols.param(a.gamma, j, 1.f, al16);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        g.p[i] = __fmul2_rn(g.p[i], gamma.p[i]);
        xh.p[i] = __fmul2_rn(__fadd2_rn(xh.p[i], make_float2(-st.x, -st.x)),
                             make_float2(st.y, st.y));
      }
    };
    float2 s1 = make_float2(0.f, 0.f), s2 = s1;
#pragma unroll 2
    for (int j = 0; cols.has(j); ++j) {
      Vals<VEC> g, xh;
      terms(j, g, xh);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        s1 = __fadd2_rn(g.p[i], s1);
        s2 = __ffma2_rn(g.p[i], xh.p[i], s2);
      }
    }
    const float2 s = block_sum(make_float2(s1.x + s1.y, s2.x + s2.y), scr);
    const float k1 = -s.x * a.rC * st.y, k2 = -s.y * a.rC * st.y;
#pragma unroll 2
    for (int j = 0; cols.has(j); ++j) {
      Vals<VEC> g, xh;
      terms(j, g, xh);
#pragma unroll
      for (int i = 0; i < NP; ++i)
        g.p[i] = __ffma2_rn(g.p[i], make_float2(st.y, st.y),
                            __ffma2_rn(xh.p[i], make_float2(k2, k2), make_float2(k1, k1)));
      cols.store(dr, j, g);
    }
  }
}

// part[slice][c] = (sum dy xh, sum dy) over the slice's rows: a unit a lane, and a slice
// of the rows a block, a warp a row of it.
constexpr int CT = 256, CWARPS = CT / 32;
template <typename TX, typename TY, int VEC>
__global__ void __launch_bounds__(CT)
k_ln_cols(LnArgs a, const TX* __restrict__ x, const TY* __restrict__ dy,
          float2* __restrict__ part, int per) {
  constexpr int NP = kPairs(VEC), CH = 2 * NP;
  __shared__ float2 scr[CWARPS][CH][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Cols<VEC> cols{(int)(blockIdx.x * 32) + lane, (int)gridDim.x * 32, a.C};
  const long long r0 = (long long)blockIdx.y * per, r1 = min((long long)a.rows, r0 + per);
  Vals<VEC> dg, db;
  dg.fill(0.f);
  db.fill(0.f);
  if (cols.has(0)) {
#pragma unroll 4
    for (long long r = r0 + warp; r < r1; r += CWARPS) {
      const Row w = row_of(a, (int)r);
      if (!w.live) continue;
      const float2 st = a.stats[r];
      const Vals<VEC> g = cols.load(dy + w.y, 0), v = cols.load(x + w.x, 0);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float2 xh = __fmul2_rn(__fadd2_rn(v.p[i], make_float2(-st.x, -st.x)),
                                     make_float2(st.y, st.y));
        dg.p[i] = __ffma2_rn(g.p[i], xh, dg.p[i]);
        db.p[i] = __fadd2_rn(g.p[i], db.p[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i)
    scr[warp][i][lane] = make_float2(i & 1 ? dg.p[i / 2].y : dg.p[i / 2].x,
                                     i & 1 ? db.p[i / 2].y : db.p[i / 2].x);
  __syncthreads();
  // a warp a channel of the units
  for (int i = warp; i < CH; i += CWARPS) {
    if (!(VEC == 1 && i ? cols.both(0) : cols.has(0))) continue;
    float2 s = scr[0][i][lane];
    for (int k = 1; k < CWARPS; ++k) s = __fadd2_rn(s, scr[k][i][lane]);
    part[(long long)blockIdx.y * a.C + cols.at(0) + (VEC == 1 ? i * cols.lanes : i)] = s;
  }
}

// dgamma, dbeta: the column sums of part [n][C], 8 channels a block, its 32 groups
// of threads 8 rows each at a time.  The sums meet in trees: at most 11 roundings on a
// row's way, up to 50 one after another (7 x 333 x 360 with the sums 6.4 us, was 6.9).
constexpr int PT = 256, PCOLS = 8, PGROUPS = PT / PCOLS, PROWS = 8;
template <int N>
__device__ __forceinline__ float2 tree(float2 (&v)[N]) {
#pragma unroll
  for (int h = N / 2; h; h >>= 1)
#pragma unroll
    for (int k = 0; k < h; ++k) v[k] = __fadd2_rn(v[k], v[k + h]);
  return v[0];
}
__global__ void __launch_bounds__(PT)
k_ln_params(const float2* __restrict__ part, int n, int C, float* __restrict__ dgamma,
            float* __restrict__ dbeta) {
  constexpr int WARPS = PT / 32;
  __shared__ float2 scr[WARPS][PCOLS];
  const int col = threadIdx.x % PCOLS, group = threadIdx.x / PCOLS;
  const int c = blockIdx.x * PCOLS + col;
  ptx::griddep_wait();
  float2 s = make_float2(0.f, 0.f), v[PROWS];
  if (c < C)
    for (int r0 = group; r0 < n; r0 += PROWS * PGROUPS) {
#pragma unroll
      for (int k = 0; k < PROWS; ++k) {
        const int r = r0 + k * PGROUPS;
        v[k] = r < n ? __ldcg(part + (long long)r * C + c) : make_float2(0.f, 0.f);
      }
      s = __fadd2_rn(s, tree(v));
    }
#pragma unroll
  for (int d = PCOLS; d < 32; d <<= 1) {
    s.x += __shfl_xor_sync(0xffffffffu, s.x, d);
    s.y += __shfl_xor_sync(0xffffffffu, s.y, d);
  }
  if ((threadIdx.x & 31) < PCOLS) scr[threadIdx.x >> 5][col] = s;
  __syncthreads();
  if (group || c >= C) return;
  float2 w[WARPS];
#pragma unroll
  for (int k = 0; k < WARPS; ++k) w[k] = scr[k][col];
  s = tree(w);
  if (dgamma) dgamma[c] = s.x;
  if (dbeta) dbeta[c] = s.y;
}

// Rows of sums that the workspace holds (it may not depend on the device), for rows that
// a team may take and for those that none does.
constexpr int PART_ROWS = 608, WIDE_ROWS = 64, WIDE = 24 * MAX_THREADS;

template <typename TX, typename TY>
struct Bwd {
  const LnArgs& a;
  const void *x, *dy;
  void* dx;
  float2* part;
  int* part_rows;
  cudaStream_t st;
  template <int VEC, int NV, int MODE>
  cudaError_t run(Team t) const {
    static Known known;
    const auto k = k_ln_bwd<TX, TY, VEC, NV, MODE>;
    if (kBound<VEC, NV, MODE> <= 256) t.teams = kBound<VEC, NV, MODE> / t.lanes;
    const int threads = t.lanes * t.teams;
    const size_t sums = sizeof(float2) * 2 * kPairs(VEC) * threads;
    const size_t smem = std::max(sums, Ring<VEC, NV, STAGES, TX>::bytes(threads) +
                                           Ring<VEC, NV, STAGES, TY>::bytes(threads));
    int per = 0;
    const cudaError_t e = blocks_per_sm(k, &known, threads, smem, &per);
    if (e != cudaSuccess) return e;
    // (two rows a team before there are more blocks, each of which leaves a row of sums: 8
    // x 200 rows of 512 7.1 us, with one 8.8; 4 x 60 of 256 5.8 and 5.3)
    const int grid = (int)std::min<long long>(
        std::min<long long>(cdiv(a.rows, 2 * t.teams), part_rows_max(a)),
        (long long)per * num_sms());
    k<<<grid, threads, smem, st>>>(a, t, (const TX*)x, (const TY*)dy, (TX*)dx, part);
    *part_rows = grid;
    return cudaGetLastError();
  }
};

template <typename TX, typename TY>
cudaError_t ln_bwd(const LnArgs& a, const void* x, const void* dy, void* dx, float2* part,
                   int* part_rows, cudaStream_t st) {
  constexpr int V16 = 16 / (int)std::max(sizeof(TX), sizeof(TY));
  const int vec = vec_of(a, sizeof(TX), x, dx, sizeof(TY), dy);
  cudaError_t e;
  // (their sums stay in registers)
  const Bwd<TX, TY> f{a, x, dy, dx, part, part_rows, st};
  if (by_team<V16, (V16 == 8 ? 24 : 16), 16, 16, 6>(a.C, vec, f, &e)) return e;
  const bool wide = vec == V16;
  const auto k = wide ? k_ln_bwd_wide<TX, TY, V16> : k_ln_bwd_wide<TX, TY, 1>;
  k<<<std::min(a.rows, 4 * num_sms()), WT, 0, st>>>(a, (const TX*)x, (const TY*)dy, (TX*)dx);
  e = cudaGetLastError();
  if (e != cudaSuccess || !part) return e;
  const int n = std::min(WIDE_ROWS, part_rows_max(a));
  const auto c = wide ? k_ln_cols<TX, TY, V16> : k_ln_cols<TX, TY, 1>;
  c<<<dim3((unsigned)cdiv(a.C, 32 * (wide ? V16 : 2)), n), CT, 0, st>>>(
      a, (const TX*)x, (const TY*)dy, part, (int)cdiv(a.rows, n));
  *part_rows = n;
  return cudaGetLastError();
}

}  // namespace

namespace ln {

int part_rows_max(const LnArgs& a) {
  return std::min(a.C > WIDE ? WIDE_ROWS : PART_ROWS, std::max(1, a.rows));
}

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
  // (its blocks come in under the sums' tail and wait for them)
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)cdiv(C, PCOLS));
  cfg.blockDim = dim3(PT);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_ln_params, part, rows, C, dgamma, dbeta);
}

}  // namespace ln
}  // namespace rnnt
