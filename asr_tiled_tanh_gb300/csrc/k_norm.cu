// k_norm.cu -- group norm with an activation over encoder frames, channels
// last (include/rnnt_ops.h).
#include <atomic>

#include "ops.h"
#include "ptx.cuh"

namespace rnnt {
namespace {

// Division of 0 <= n < 2^31 by a fixed d (round-up reciprocal): a multiply-high,
// an add and a shift in place of the twenty instructions of a 32-bit division.
struct FastDiv {
  uint32_t d, mul, shift;
};
FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((1ull << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
  return f;
}
__device__ __forceinline__ int operator/(int n, const FastDiv& f) {
  return (int)((__umulhi((uint32_t)n, f.mul) + (uint32_t)n) >> f.shift);
}

struct NormArgs {
  int B, T, C, G, cg, act;
  FastDiv cg_div;
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

// ---- activation -------------------------------------------------------------
// sigmoid of two values.  fp32: to fp32's own accuracy.  bf16: ex2 and one
// reciprocal for the pair, 1 / (p q) times q and p (three special-function
// operations instead of four, which is what bounds the bf16 kernels next to
// their memory traffic); the exponent is capped at 60 so that p q stays finite
// (sigmoid below 2^-60 is taken as that).
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2 u) {
  if constexpr (sizeof(T) == 4) {
    return make_float2(1.f / (1.f + expf(-u.x)), 1.f / (1.f + expf(-u.y)));
  } else {
    const float kL = -1.4426950408889634f;
    const float2 t = __fmul2_rn(u, make_float2(kL, kL));
    const float2 pq = __fadd2_rn(make_float2(ptx::ex2(fminf(t.x, 60.f)),
                                             ptx::ex2(fminf(t.y, 60.f))),
                                 make_float2(1.f, 1.f));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(pq.x * pq.y));
    return __fmul2_rn(make_float2(pq.y, pq.x), make_float2(r, r));
  }
}

template <int ACT, typename T>
__device__ __forceinline__ float2 act2(float2 u) {
  if constexpr (ACT == RNNT_ACT_SILU) return __fmul2_rn(u, sigmoid2<T>(u));
  if constexpr (ACT == RNNT_ACT_RELU)  // (NaN stays NaN)
    return make_float2(u.x < 0.f ? 0.f : u.x, u.y < 0.f ? 0.f : u.y);
  return u;
}

// dy act'(u)
template <int ACT, typename T>
__device__ __forceinline__ float2 dact2(float2 dy, float2 u) {
  if constexpr (ACT == RNNT_ACT_SILU) {
    const float2 s = sigmoid2<T>(u);
    // s + u s (1 - s) = s + (u s) - (u s) s
    const float2 us = __fmul2_rn(u, s);
    const float2 d = __fadd2_rn(s, __ffma2_rn(make_float2(-us.x, -us.y), s, us));
    return __fmul2_rn(dy, d);
  }
  if constexpr (ACT == RNNT_ACT_RELU)
    return make_float2(u.x > 0.f ? dy.x : 0.f, u.y > 0.f ? dy.y : 0.f);
  return dy;
}

// ---- vectors ------------------------------------------------------------------
// A thread's VEC (4 or 1) consecutive channels of a frame, as pairs of fp32.
template <int VEC>
struct Ch {
  float2 v[VEC == 4 ? 2 : 1];
};
constexpr int kPairs(int vec) { return vec == 4 ? 2 : 1; }

template <int VEC, typename T>
__device__ __forceinline__ Ch<VEC> load_ch(const T* p) {
  Ch<VEC> c;
  if constexpr (VEC == 1) {
    c.v[0] = make_float2(to_f<T>(*p), 0.f);
  } else if constexpr (sizeof(T) == 4) {
    const float4 q = *(const float4*)p;
    c.v[0] = make_float2(q.x, q.y);
    c.v[1] = make_float2(q.z, q.w);
  } else {
    const uint2 q = *(const uint2*)p;
    c.v[0] = make_float2(ptx::bf16lo(q.x), ptx::bf16hi(q.x));
    c.v[1] = make_float2(ptx::bf16lo(q.y), ptx::bf16hi(q.y));
  }
  return c;
}
template <int VEC, typename T>
__device__ __forceinline__ void store_ch(T* p, const Ch<VEC>& c) {
  if constexpr (VEC == 1) {
    *p = from_f<T>(c.v[0].x);
  } else if constexpr (sizeof(T) == 4) {
    *(float4*)p = make_float4(c.v[0].x, c.v[0].y, c.v[1].x, c.v[1].y);
  } else {
    *(uint2*)p = make_uint2(ptx::pack_bf16x2(c.v[0].x, c.v[0].y),
                            ptx::pack_bf16x2(c.v[1].x, c.v[1].y));
  }
}

// ---- slabs ----------------------------------------------------------------------
// A slab is one sample's frames of kk whole groups (W = kk C/G channels, at
// least 64 bytes of a frame where the groups allow).  A cluster of S blocks
// owns it, a contiguous share of its frames each; RES blocks copy their share
// into shared memory once and make every pass over it there, so that x (and
// dy) are read once from DRAM and y (dx) written once, which is the kernels'
// bound.  Shares are kept to 72 KB so that three blocks share an SM: one
// computes while the others' copies are in flight.  Slabs that eight blocks
// cannot hold, and rows that are not 16-byte aligned, are read from global
// memory in every pass (RES = 0).
constexpr int NT = 256, NWARPS = NT / 32;
constexpr int MAX_KK = 128;
constexpr int SHARE = 72 * 1024, SHARE_MAX = 208 * 1024;

struct Slab {
  int kk, W, S;      // groups and channels per slab, blocks per slab
  int per_max;       // frames a block may own
  int cbv;           // vectors of a column block (all VEC-wide columns of W, at most NT)
  int pow2;          // cbv is a power of two <= 32: columns meet by shuffles first
  int scratch;       // scratch bytes per reduced quantity
  FastDiv per_sample_div, S_div, cbv_div;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// value at the same shared address of another block of the cluster
__device__ __forceinline__ float peer_f32(const float* p, int rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// Sums over the block's frames of NA quantities per channel, for the channels
// of the current column block: afterwards res[q * n + c], n = cbv * VEC, where
// res is returned (behind the NA * rows * n partial sums).
template <int NA, int VEC>
__device__ __forceinline__ const float* reduce_channels(const Slab& sl,
                                                        float2 (&acc)[NA][kPairs(VEC)],
                                                        float* scr, int col, int rg, bool active) {
  const int n = sl.cbv * VEC, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = sl.pow2 ? NWARPS : NT / sl.cbv_div;
  if (sl.pow2) {
    for (int o = sl.cbv; o < 32; o <<= 1) {
#pragma unroll
      for (int q = 0; q < NA; ++q)
#pragma unroll
        for (int i = 0; i < kPairs(VEC); ++i) {
          acc[q][i].x += __shfl_xor_sync(0xffffffffu, acc[q][i].x, o);
          if (VEC > 1) acc[q][i].y += __shfl_xor_sync(0xffffffffu, acc[q][i].y, o);
        }
    }
    rg = warp;
    active = lane < sl.cbv;
  }
  if (active) {
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      float* d = scr + (q * rows + rg) * n + col * VEC;
#pragma unroll
      for (int i = 0; i < kPairs(VEC); ++i) {
        d[2 * i] = acc[q][i].x;
        if (VEC > 1) d[2 * i + 1] = acc[q][i].y;
      }
    }
  }
  __syncthreads();
  float* res = scr + NA * rows * n;
  for (int c = threadIdx.x; c < NA * n; c += NT) {
    const int q = NA > 1 && c >= n;
    const float* d = scr + q * (rows - 1) * n + c;
    float t = 0.f;
#pragma unroll 8
    for (int r = 0; r < rows; ++r) t += d[r * n];
    res[c] = t;
  }
  __syncthreads();
  return res;
}

// gs[q][g] += sum over the group's channels of the column block of w(c) scr[q][c]
template <int NA, int VEC, typename F>
__device__ __forceinline__ void reduce_groups(const Slab& sl, int cg, int cb, const float* scr,
                                              float (*gs)[MAX_KK], F w) {
  const int n = sl.cbv * VEC, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int g = warp; g < sl.kk; g += NWARPS) {
    const int c0 = max(g * cg, cb), c1 = min(min((g + 1) * cg, cb + n), sl.W);
    float s[NA] = {};
    for (int c = c0 + lane; c < c1; c += 32)
#pragma unroll
      for (int q = 0; q < NA; ++q) s[q] += w(c) * scr[(size_t)q * n + c - cb];
#pragma unroll
    for (int q = 0; q < NA; ++q) {
#pragma unroll
      for (int o = 16; o; o >>= 1) s[q] += __shfl_xor_sync(0xffffffffu, s[q], o);
      if (lane == 0) gs[q][g] += s[q];
    }
  }
}

// The block's frames of a slab, copied to shared memory as dense rows of W.
template <typename T>
__device__ __forceinline__ void copy_share(T* dst, const T* src, long long ld, int rows, int W) {
  const int cpr = W * (int)sizeof(T) / 16;  // 16-byte pieces of a row
  const int per = NT / cpr;                 // rows per step of the block (cpr <= NT)
  if (per > 0) {
    const int r0 = threadIdx.x / cpr, c = threadIdx.x - r0 * cpr;
    if (r0 >= per) return;
    const char* g = (const char*)(src + r0 * ld) + 16 * c;
    uint32_t d = ptx::smem_u32(dst) + (uint32_t)(r0 * cpr + c) * 16;
    for (int r = r0; r < rows; r += per) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(g) : "memory");
      g += (long long)per * ld * sizeof(T);
      d += (uint32_t)(per * cpr) * 16;
    }
  } else {
    for (int i = threadIdx.x; i < rows * cpr; i += NT) {
      const int r = i / cpr, c = i - r * cpr;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst) + 16 * i),
                   "l"((const char*)(src + r * ld) + 16 * c)
                   : "memory");
    }
  }
}
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
}

// The block's slab, frames and column.
template <int VEC>
struct Where {
  int b, c0, rank, tb, t0, rows, v, rg, step;
  bool active;
};
template <int VEC>
__device__ __forceinline__ Where<VEC> where(const NormArgs& a, const Slab& sl) {
  Where<VEC> w;
  const int slab = (int)blockIdx.x / sl.S_div;
  w.rank = blockIdx.x - slab * sl.S;
  w.b = slab / sl.per_sample_div;
  w.c0 = (slab - w.b * (int)sl.per_sample_div.d) * sl.W;
  w.tb = frames_of(a, w.b);
  const int per = (w.tb + sl.S - 1) / sl.S_div;
  w.t0 = min(w.tb, w.rank * per);
  w.rows = min(w.tb, w.t0 + per) - w.t0;
  w.rg = (int)threadIdx.x / sl.cbv_div;
  w.v = threadIdx.x - w.rg * sl.cbv;
  w.step = NT / sl.cbv_div;
  w.active = w.rg < w.step;
  return w;
}

// zeros in the block's share of the frames past the sample's length
template <int VEC, typename T>
__device__ __forceinline__ void zero_tail(const NormArgs& a, const Slab& sl, const Where<VEC>& w,
                                          T* out, long long ld) {
  const int left = a.T - w.tb, per = (left + sl.S - 1) / sl.S_div;
  const int z0 = w.tb + min(left, w.rank * per), z1 = w.tb + min(left, (w.rank + 1) * per);
  if (!w.active) return;
  const Ch<VEC> z{};
  for (int cb = 0; cb < sl.W; cb += sl.cbv * VEC) {
    const int c = cb + w.v * VEC;
    if (c >= sl.W) continue;
    T* p = out + (long long)(z0 + w.rg) * ld + c;
    const long long inc = w.step * ld;
#pragma unroll 4
    for (int t = z0 + w.rg; t < z1; t += w.step, p += inc) store_ch<VEC, T>(p, z);
  }
}

// Frames of the calling thread's column: rg, rg + step, ...
template <int VEC>
__device__ __forceinline__ int rows_of(const Where<VEC>& w) {
  return w.active && w.rg < w.rows ? (w.rows - 1 - w.rg) / w.step + 1 : 0;
}

// Row steps: within shared memory 32 bits do.
template <int RES> struct StepType { using type = long long; };
template <> struct StepType<1> { using type = int; };

template <typename T, int VEC, int ACT, int RES>
__global__ void __launch_bounds__(NT, 3)
k_norm_fwd(NormArgs a, Slab sl, const T* __restrict__ x, T* __restrict__ y) {
  extern __shared__ __align__(16) unsigned char smem[];
  // (gs[1], mean_s and n_s are read by the cluster's other blocks)
  __shared__ float gs[2][MAX_KK], mean_s[MAX_KK], n_s;
  __shared__ float mean_t[MAX_KK], rstd_t[MAX_KK];
  T* tile = (T*)smem;
  float* scr = (float*)(smem + (RES ? align_up((size_t)sl.per_max * sl.W * sizeof(T), 16) : 0));
  const Where<VEC> w = where<VEC>(a, sl);
  const T* xs = x + w.b * a.xb + w.c0;
  T* ys = y + w.b * a.yb + w.c0;
  if (RES) copy_share(tile, xs + (long long)w.t0 * a.xf, a.xf, w.rows, sl.W);
  zero_tail<VEC, T>(a, sl, w, ys, a.yf);
  using Step = typename StepType<RES>::type;
  const T* src = RES ? tile : xs + (long long)w.t0 * a.xf;
  const Step ld = RES ? sl.W : a.xf, inc = ld * w.step;
  const int nb = sl.cbv * VEC, cnt = rows_of(w);
  const float n = (float)w.rows * a.cg;
  if (threadIdx.x < sl.kk) gs[0][threadIdx.x] = gs[1][threadIdx.x] = 0.f;
  if (RES) copy_wait();
  __syncthreads();
  // One pass over the data: every thread sums its own frames of a channel and
  // their squares about the first of them (its few frames lose no digits to
  // that, wherever the mean is).  Then the block's mean, and the squares about
  // that: q - s^2 / k about the thread's mean, plus k (its mean - mean)^2.
  float2 fsum[kPairs(VEC)], fsq[kPairs(VEC)];
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
#pragma unroll 1
    for (int cb = 0; cb < sl.W; cb += nb) {
      const int c = cb + w.v * VEC;
      const bool on = w.active && c < sl.W && cnt > 0;
      float2 acc[1][kPairs(VEC)] = {};
      // (a slab of one column block keeps its sums; wider ones read again)
      if (on && (half == 0 || nb < sl.W)) {
        const T* p = src + w.rg * ld + c;
        const Ch<VEC> first = load_ch<VEC, T>(p);
        float2 m[kPairs(VEC)], s0[kPairs(VEC)] = {}, q0[kPairs(VEC)] = {};
#pragma unroll
        for (int i = 0; i < kPairs(VEC); ++i)
          m[i] = make_float2(-first.v[i].x, -first.v[i].y);
#pragma unroll 4
        for (int k = 0; k < cnt; ++k, p += inc) {
          const Ch<VEC> q = load_ch<VEC, T>(p);
#pragma unroll
          for (int i = 0; i < kPairs(VEC); ++i) {
            const float2 d = __fadd2_rn(q.v[i], m[i]);
            s0[i] = __fadd2_rn(s0[i], d);
            q0[i] = __ffma2_rn(d, d, q0[i]);
          }
        }
        const float k = (float)cnt, rk = 1.f / k;
#pragma unroll
        for (int i = 0; i < kPairs(VEC); ++i) {
          const float2 mk = __fmul2_rn(s0[i], make_float2(rk, rk));
          fsum[i] = __fadd2_rn(mk, first.v[i]);
          fsq[i] = __ffma2_rn(make_float2(-s0[i].x, -s0[i].y), mk, q0[i]);
        }
      }
      if (on) {
        const float2 k = make_float2((float)cnt, (float)cnt);
#pragma unroll
        for (int i = 0; i < kPairs(VEC); ++i) {
          if (half == 0) {
            acc[0][i] = __fmul2_rn(k, fsum[i]);
          } else {
            const int ca = c + 2 * i, cz = VEC > 1 ? ca + 1 : ca;
            const float2 d = __fadd2_rn(fsum[i], make_float2(-mean_s[ca / a.cg_div],
                                                             -mean_s[cz / a.cg_div]));
            acc[0][i] = __ffma2_rn(__fmul2_rn(d, d), k, fsq[i]);
          }
        }
      }
      const float* res =
          reduce_channels<1, VEC>(sl, acc, scr, w.v, w.rg, w.active && c < sl.W);
      reduce_groups<1, VEC>(sl, a.cg, cb, res, gs + half, [](int) { return 1.f; });
    }
    __syncthreads();
    if (half == 0) {
      for (int g = threadIdx.x; g < sl.kk; g += NT) mean_s[g] = w.rows ? gs[0][g] / n : 0.f;
      if (threadIdx.x == 0) n_s = n;
      __syncthreads();
    }
  }
  const float* m2_s = gs[1];
  // the blocks' (n, mean, M2) joined in order
  if (sl.S > 1) {
    cluster_arrive();
    cluster_wait();
  }
  for (int g = threadIdx.x; g < sl.kk; g += NT) {
    float nt = 0.f, mt = 0.f, st = 0.f;
    for (int k = 0; k < sl.S; ++k) {
      const float nk = sl.S > 1 ? peer_f32(&n_s, k) : n_s;
      if (nk == 0.f) continue;
      const float mk = sl.S > 1 ? peer_f32(&mean_s[g], k) : mean_s[g];
      const float sk = sl.S > 1 ? peer_f32(&m2_s[g], k) : m2_s[g];
      const float d = mk - mt, all = nt + nk, f = nk / all;
      mt += d * f;
      st += sk + d * d * (nt * f);
      nt = all;
    }
    const float rstd = nt > 0.f ? 1.f / sqrtf(st / nt + a.eps) : 0.f;
    mean_t[g] = mt;
    rstd_t[g] = rstd;
    if (w.rank == 0) a.stats[(long long)w.b * a.G + w.c0 / a.cg + g] = make_float2(mt, rstd);
  }
  __syncthreads();
  if (sl.S > 1) cluster_arrive();  // (waited for at the end: peers may still read)
  T* yt = ys + (long long)w.t0 * a.yf;
#pragma unroll 1
  for (int cb = 0; cb < sl.W; cb += nb) {
    const int c = cb + w.v * VEC;
    if (!w.active || c >= sl.W) continue;
    if (cnt == 0) continue;
    float2 m[kPairs(VEC)], s[kPairs(VEC)], be[kPairs(VEC)];
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) {
      float2 rs, ga;
      const int ca = c + 2 * i, cz = VEC > 1 ? ca + 1 : ca;
      const int gx = ca / a.cg_div, gz = cz / a.cg_div;
      m[i] = make_float2(-mean_t[gx], -mean_t[gz]);
      rs = make_float2(rstd_t[gx], rstd_t[gz]);
      ga = a.gamma ? make_float2(a.gamma[w.c0 + ca], a.gamma[w.c0 + cz]) : make_float2(1.f, 1.f);
      be[i] = a.beta ? make_float2(a.beta[w.c0 + ca], a.beta[w.c0 + cz]) : make_float2(0.f, 0.f);
      s[i] = __fmul2_rn(rs, ga);
    }
    const T* p = src + w.rg * ld + c;
    T* o = yt + w.rg * a.yf + c;
    const long long oinc = w.step * a.yf;
#pragma unroll 4
    for (int k = 0; k < cnt; ++k, p += inc, o += oinc) {
      Ch<VEC> q = load_ch<VEC, T>(p);
#pragma unroll
      for (int i = 0; i < kPairs(VEC); ++i)
        q.v[i] = act2<ACT, T>(__ffma2_rn(__fadd2_rn(q.v[i], m[i]), s[i], be[i]));
      store_ch<VEC, T>(o, q);
    }
  }
  __syncwarp();
  if (sl.S > 1) cluster_wait();
}

// part: per slab block and channel (sum g xh, sum g), [B][S][C].
template <typename T, int VEC, int ACT, int RES>
__global__ void __launch_bounds__(NT, RES ? 3 : 2)
k_norm_bwd(NormArgs a, Slab sl, const T* __restrict__ x, const T* __restrict__ dy,
           T* __restrict__ dx, float2* __restrict__ part) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float gs[2][MAX_KK];  // read by the cluster's other blocks
  __shared__ float m1_t[MAX_KK], m2_t[MAX_KK];
  const size_t tb = RES ? align_up((size_t)sl.per_max * sl.W * sizeof(T), 16) : 0;
  T *tx = (T*)smem, *td = (T*)(smem + tb);
  float* scr = (float*)(smem + 2 * tb);
  const Where<VEC> w = where<VEC>(a, sl);
  const T* xs = x + w.b * a.xb + w.c0 + (long long)w.t0 * a.xf;
  const T* ds = dy + w.b * a.yb + w.c0 + (long long)w.t0 * a.yf;
  T* os = dx + w.b * a.xb + w.c0;
  if (RES) {
    copy_share(tx, xs, a.xf, w.rows, sl.W);
    copy_share(td, ds, a.yf, w.rows, sl.W);
  }
  zero_tail<VEC, T>(a, sl, w, os, a.xf);
  os += (long long)w.t0 * a.xf;
  const T *sx = RES ? tx : xs, *sd = RES ? td : ds;
  using Step = typename StepType<RES>::type;
  const Step lx = RES ? sl.W : a.xf, ldy = RES ? sl.W : a.yf;
  const Step xinc = lx * w.step, dinc = ldy * w.step;
  const int nb = sl.cbv * VEC, cnt = rows_of(w);
  const float2* stats = a.stats + (long long)w.b * a.G + w.c0 / a.cg;
  for (int g = threadIdx.x; g < sl.kk; g += NT) gs[0][g] = gs[1][g] = 0.f;
  if (RES) copy_wait();
  __syncthreads();
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int cb = 0; cb < sl.W; cb += nb) {
      const int c = cb + w.v * VEC;
      const bool on = w.active && c < sl.W;
      float2 m[kPairs(VEC)], rs[kPairs(VEC)], ga[kPairs(VEC)], be[kPairs(VEC)];
      if (on) {
#pragma unroll
        for (int i = 0; i < kPairs(VEC); ++i) {
          const int ca = c + 2 * i, cz = VEC > 1 ? ca + 1 : ca;
          const float2 p = stats[ca / a.cg_div], q = stats[cz / a.cg_div];
          m[i] = make_float2(-p.x, -q.x);
          rs[i] = make_float2(p.y, q.y);
          ga[i] = a.gamma ? make_float2(a.gamma[w.c0 + ca], a.gamma[w.c0 + cz])
                          : make_float2(1.f, 1.f);
          be[i] = a.beta ? make_float2(a.beta[w.c0 + ca], a.beta[w.c0 + cz])
                         : make_float2(0.f, 0.f);
        }
      }
      if (pass == 0) {
        float2 acc[2][kPairs(VEC)] = {};
        if (on) {
          const T *px = sx + w.rg * lx + c, *pd = sd + w.rg * ldy + c;
#pragma unroll 2
          for (int k = 0; k < cnt; ++k, px += xinc, pd += dinc) {
            const Ch<VEC> q = load_ch<VEC, T>(px), d = load_ch<VEC, T>(pd);
#pragma unroll
            for (int i = 0; i < kPairs(VEC); ++i) {
              const float2 xh = __fmul2_rn(__fadd2_rn(q.v[i], m[i]), rs[i]);
              const float2 g = dact2<ACT, T>(d.v[i], __ffma2_rn(xh, ga[i], be[i]));
              acc[0][i] = __ffma2_rn(g, xh, acc[0][i]);
              acc[1][i] = __fadd2_rn(acc[1][i], g);
            }
          }
        }
        const float* res = reduce_channels<2, VEC>(sl, acc, scr, w.v, w.rg, on);
        for (int k = threadIdx.x; k < nb && cb + k < sl.W; k += NT)
          part[((long long)w.b * sl.S + w.rank) * a.C + w.c0 + cb + k] =
              make_float2(res[k], res[nb + k]);
        reduce_groups<2, VEC>(sl, a.cg, cb, res, gs, [&](int ch) {
          return a.gamma ? a.gamma[w.c0 + ch] : 1.f;
        });
      } else if (on) {
        float2 k1[kPairs(VEC)], k2[kPairs(VEC)];
#pragma unroll
        for (int i = 0; i < kPairs(VEC); ++i) {
          const int ca = c + 2 * i, gx = ca / a.cg_div, gz = (VEC > 1 ? ca + 1 : ca) / a.cg_div;
          k1[i] = make_float2(-m1_t[gx], -m1_t[gz]);
          k2[i] = make_float2(-m2_t[gx], -m2_t[gz]);
        }
        const T *px = sx + w.rg * lx + c, *pd = sd + w.rg * ldy + c;
        T* po = os + w.rg * a.xf + c;
        const long long oinc = w.step * a.xf;
#pragma unroll 2
        for (int k = 0; k < cnt; ++k, px += xinc, pd += dinc, po += oinc) {
          const Ch<VEC> q = load_ch<VEC, T>(px), d = load_ch<VEC, T>(pd);
          Ch<VEC> o;
#pragma unroll
          for (int i = 0; i < kPairs(VEC); ++i) {
            const float2 xh = __fmul2_rn(__fadd2_rn(q.v[i], m[i]), rs[i]);
            const float2 g = dact2<ACT, T>(d.v[i], __ffma2_rn(xh, ga[i], be[i]));
            o.v[i] = __fmul2_rn(rs[i], __ffma2_rn(xh, k2[i], __ffma2_rn(g, ga[i], k1[i])));
          }
          store_ch<VEC, T>(po, o);
        }
      }
    }
    if (pass) break;
    __syncthreads();
    if (sl.S > 1) {
      cluster_arrive();
      cluster_wait();
    }
    const float n = (float)w.tb * a.cg;
    for (int g = threadIdx.x; g < sl.kk; g += NT) {
      float s2 = 0.f, s1 = 0.f;
      for (int k = 0; k < sl.S; ++k) {
        s2 += sl.S > 1 ? peer_f32(&gs[0][g], k) : gs[0][g];
        s1 += sl.S > 1 ? peer_f32(&gs[1][g], k) : gs[1][g];
      }
      m1_t[g] = n > 0.f ? s1 / n : 0.f;
      m2_t[g] = n > 0.f ? s2 / n : 0.f;
    }
    __syncthreads();
    if (sl.S > 1) cluster_arrive();  // (waited for at the end: peers may still read)
  }
  __syncwarp();
  if (sl.S > 1) cluster_wait();
}

// dgamma, dbeta: the column sums of part [rows][C], 32 channels a cluster, a
// contiguous share of the rows per block, the blocks' sums joined in order.
__global__ void __launch_bounds__(NT)
k_norm_params(const float2* __restrict__ part, int rows, int C, int S, float* __restrict__ dgamma,
              float* __restrict__ dbeta) {
  __shared__ float2 ws[NWARPS][32];
  __shared__ float tot[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % S, c = (blockIdx.x / S) * 32 + lane;
  const int per = (rows + S - 1) / S, r1 = min(rows, (rank + 1) * per);
  float2 s = make_float2(0.f, 0.f);
  if (c < C) {
#pragma unroll 4
    for (int r = rank * per + warp; r < r1; r += NWARPS)
      s = __fadd2_rn(s, __ldg(part + (long long)r * C + c));
  }
  ws[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    for (int k = 1; k < NWARPS; ++k) s = __fadd2_rn(s, ws[k][lane]);
    tot[0][lane] = s.x;
    tot[1][lane] = s.y;
  }
  __syncthreads();
  if (S > 1) {
    cluster_arrive();
    cluster_wait();
  }
  if (rank == 0 && warp == 0 && c < C) {
    for (int k = 1; k < S; ++k)
      s = __fadd2_rn(s, make_float2(peer_f32(&tot[0][lane], k), peer_f32(&tot[1][lane], k)));
    if (dgamma) dgamma[c] = s.x;
    if (dbeta) dbeta[c] = s.y;
  }
  __syncwarp();
  if (S > 1) {
    cluster_arrive();
    cluster_wait();
  }
}

bool norm_args(const rnnt_norm_dims* d, NormArgs* a) {
  if (!d || d->B < 0 || d->T < 1 || d->C < 1 || d->G < 1 || d->C % d->G) return false;
  if (d->T > (1 << 20) || (long long)d->B * d->G > (1LL << 27)) return false;
  if (d->act < RNNT_ACT_NONE || d->act > RNNT_ACT_RELU || !op_dtype(d->dtype)) return false;
  if (!(d->eps >= 0.f)) return false;
  a->B = d->B; a->T = d->T; a->C = d->C; a->G = d->G; a->cg = d->C / d->G;
  a->act = d->act; a->eps = d->eps;
  a->cg_div = fast_div(a->cg);
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

// How a call cuts its slabs.
struct NormCut {
  Slab sl;
  int vec, res;
  size_t smem;
};

NormCut norm_cut(const NormArgs& a, int e, int tiles, bool aligned) {
  NormCut n{};
  n.vec = 0;
  // the fewest whole groups that make 64-byte pieces of a frame (16-byte
  // aligned ones); short of that, 32 channels of any alignment
  int kk = 0;
  if (aligned)
    for (int k = 1; k <= a.G && k <= MAX_KK; ++k)
      if (a.G % k == 0 && (long long)k * a.cg * e % 16 == 0) {
        kk = k;
        n.vec = 4;
        if (k * a.cg * e >= 64) break;
      }
  if (!kk) {
    n.vec = 1;
    for (int k = 1; k <= a.G && k <= MAX_KK; ++k)
      if (a.G % k == 0) {
        kk = k;
        if (k * a.cg >= 32) break;
      }
  }
  Slab& s = n.sl;
  s.kk = kk;
  s.W = kk * a.cg;
  const long long frame = (long long)s.W * e * tiles, slabs = (long long)a.B * (a.G / kk);
  s.S = 1;
  while (s.S < 8 && cdiv(a.T, s.S) * frame > SHARE) s.S *= 2;
  // few slabs: shares of at least 64 frames, until there are two blocks an SM
  while (s.S < 8 && slabs * s.S < 2 * 152 && a.T >= 128 * s.S) s.S *= 2;
  s.per_max = (int)cdiv(a.T, s.S);
  const int vr = s.W / n.vec;
  s.cbv = vr < NT ? vr : NT;
  s.pow2 = s.cbv <= 32 && (s.cbv & (s.cbv - 1)) == 0;
  const int rows = s.pow2 ? NWARPS : NT / s.cbv;
  s.scratch = 4 * (rows + 1) * s.cbv * n.vec;
  s.per_sample_div = fast_div(a.G / kk);
  s.S_div = fast_div(s.S);
  s.cbv_div = fast_div(s.cbv);
  const size_t tile = align_up((size_t)s.per_max * s.W * e, 16) * tiles;
  n.res = n.vec == 4 && tile <= SHARE_MAX;
  n.smem = (n.res ? tile : 0) + (size_t)s.scratch * tiles;
  return n;
}

// Launch a kernel in clusters of S blocks.
template <typename... KA, typename... A>
cudaError_t launch_cluster(void (*k)(KA...), unsigned grid, int S, size_t smem, cudaStream_t st,
                           A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = S;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = S > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// Shared memory above 48 KB is asked for once per kernel and device.
template <typename K>
cudaError_t opt_in(K k, std::atomic<bool>* done) {
  std::atomic<bool>& d = done[device_slot()];
  if (d.load()) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             SHARE_MAX + 16 * 1024);
  if (e == cudaSuccess) d.store(true);
  return e;
}

template <typename T, int VEC, int ACT, int RES>
cudaError_t norm_launch(const NormArgs& a, const NormCut& n, const void* x, const void* dy,
                        void* out, float2* part, cudaStream_t st) {
  static std::atomic<bool> f[kDeviceSlots], b[kDeviceSlots];
  const unsigned grid = (unsigned)((long long)a.B * (a.G / n.sl.kk) * n.sl.S);
  cudaError_t e = dy ? opt_in(k_norm_bwd<T, VEC, ACT, RES>, b)
                     : opt_in(k_norm_fwd<T, VEC, ACT, RES>, f);
  if (e != cudaSuccess) return e;
  if (dy)
    return launch_cluster(k_norm_bwd<T, VEC, ACT, RES>, grid, n.sl.S, n.smem, st, a, n.sl,
                          (const T*)x, (const T*)dy, (T*)out, part);
  return launch_cluster(k_norm_fwd<T, VEC, ACT, RES>, grid, n.sl.S, n.smem, st, a, n.sl,
                        (const T*)x, (T*)out);
}

template <typename T, int ACT>
cudaError_t norm_launch_cut(const NormArgs& a, const NormCut& n, const void* x, const void* dy,
                            void* out, float2* part, cudaStream_t st) {
  if (n.res) return norm_launch<T, 4, ACT, 1>(a, n, x, dy, out, part, st);
  if (n.vec == 4) return norm_launch<T, 4, ACT, 0>(a, n, x, dy, out, part, st);
  return norm_launch<T, 1, ACT, 0>(a, n, x, dy, out, part, st);
}

// dy NULL: forward, x -> out = y; else backward, (x, dy) -> out = dx and part.
template <typename T>
cudaError_t norm_launch_act(const NormArgs& a, const NormCut& n, const void* x, const void* dy,
                            void* out, float2* part, cudaStream_t st) {
  switch (a.act) {
    case RNNT_ACT_SILU: return norm_launch_cut<T, RNNT_ACT_SILU>(a, n, x, dy, out, part, st);
    case RNNT_ACT_RELU: return norm_launch_cut<T, RNNT_ACT_RELU>(a, n, x, dy, out, part, st);
    default: return norm_launch_cut<T, RNNT_ACT_NONE>(a, n, x, dy, out, part, st);
  }
}

// Rows that 16-byte copies and 4-element stores may take: x and dx, y and dy.
bool norm_aligned(const NormArgs& a, int e, const void* x, const void* y, const void* dx) {
  const int v = 16 / e;
  return aligned_to(x, 16) && aligned_to(y, 16) && aligned_to(dx, 16) && a.xf % v == 0 &&
         a.xb % v == 0 && a.yf % v == 0 && a.yb % v == 0;
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
  return norm_args(dims, &a) ? align_up(8 * 8 * (size_t)a.B * a.C + 8) : 0;  // up to 8 blocks a slab
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
  const int e = op_size(dims->dtype);
  const NormCut n = norm_cut(a, e, 1, norm_aligned(a, e, x, y, nullptr));
  OPS_CHECK(e == 4 ? norm_launch_act<float>(a, n, x, nullptr, y, nullptr, st)
                   : norm_launch_act<__nv_bfloat16>(a, n, x, nullptr, y, nullptr, st));
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
  const int e = op_size(dims->dtype);
  const NormCut n = norm_cut(a, e, 2, norm_aligned(a, e, x, dy, dx));
  if (a.B > 0) {
    ProfScope ps("norm_bwd", st);
    OPS_CHECK(e == 4 ? norm_launch_act<float>(a, n, x, dy, dx, part, st)
                     : norm_launch_act<__nv_bfloat16>(a, n, x, dy, dx, part, st));
  }
  if (!dgamma && !dbeta) return RNNT_OK;
  const int rows = a.B * n.sl.S, S = rows > 256 ? 8 : 1;
  OPS_LAUNCH("norm_params", launch_cluster(k_norm_params, (unsigned)cdiv(a.C, 32) * S, S, 0, st,
                                           (const float2*)part, rows, a.C, S, dgamma, dbeta));
  return RNNT_OK;
}

}  // extern "C"
