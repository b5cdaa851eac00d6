// k_norm.cu -- group norm with an activation over encoder frames, channels
// last (include/rnnt_ops.h).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "ops.h"
#include "ptx.cuh"

namespace rnnt {
namespace {

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

__device__ __forceinline__ int length_of(const NormArgs& a, int b) {
  return a.T_len ? __ldg(a.T_len + b) : a.T;
}
__device__ __forceinline__ int frames_of(const NormArgs& a, int t) {
  if (t < 0 || t > a.T) {
    report(a.status, RNNT_ERR_LENGTH_RANGE);
    return 0;
  }
  return t;
}

// ---- activation -------------------------------------------------------------
// sigmoid of two values by the special-function unit's ex2 and reciprocal
// (relative error about 2^-22; a large negative u gives 1 / inf = 0).  fp32 also
// carries what the product u log2(e) rounds off, or large |u| would lose digits
// in the exponent; expf and a division, 30 instructions for these 8, held the
// fp32 kernels to half the bandwidth.
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2 u) {
  const float kL = -1.4426950408889634f;
  const float2 t = __fmul2_rn(u, make_float2(kL, kL));
  float2 e = make_float2(ptx::ex2(t.x), ptx::ex2(t.y));
  if constexpr (sizeof(T) == 4) {
    // -log2(e) = kL + kLow; 2^(t + f) = 2^t (1 + f ln 2)
    const float kLow = (float)(-1.4426950408889634 - (double)kL), kLn2 = 0.6931471805599453f;
    const float2 f = __ffma2_rn(u, make_float2(kLow, kLow),
                                __ffma2_rn(u, make_float2(kL, kL), make_float2(-t.x, -t.y)));
    const float2 c = __ffma2_rn(f, make_float2(kLn2, kLn2), make_float2(1.f, 1.f));
    // (beyond, e is 0 or so large that only 1 or 0 is left, and f may be NaN)
    e = make_float2(fabsf(t.x) < 126.f ? e.x * c.x : e.x, fabsf(t.y) < 126.f ? e.y * c.y : e.y);
  }
  const float2 p = __fadd2_rn(e, make_float2(1.f, 1.f));
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(p.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(p.y));
  return r;
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
// A thread's VEC (8, 4, 2 or 1) consecutive channels of a frame, as pairs of fp32.
constexpr int kPairs(int vec) { return vec == 1 ? 1 : vec / 2; }
template <int VEC>
struct Ch {
  float2 v[kPairs(VEC)];
};

template <int VEC, typename T>
__device__ __forceinline__ Ch<VEC> load_ch(const T* p) {
  Ch<VEC> c;
  if constexpr (VEC == 1) {
    c.v[0] = make_float2(to_f<T>(*p), 0.f);
  } else if constexpr (VEC == 2 && sizeof(T) == 4) {
    c.v[0] = *(const float2*)p;
  } else if constexpr (VEC == 2) {
    const uint32_t q = *(const uint32_t*)p;
    c.v[0] = make_float2(ptx::bf16lo(q), ptx::bf16hi(q));
  } else if constexpr (sizeof(T) == 4) {
    const float4 q = *(const float4*)p;
    c.v[0] = make_float2(q.x, q.y);
    c.v[1] = make_float2(q.z, q.w);
  } else if constexpr (VEC == 4) {
    const uint2 q = *(const uint2*)p;
    c.v[0] = make_float2(ptx::bf16lo(q.x), ptx::bf16hi(q.x));
    c.v[1] = make_float2(ptx::bf16lo(q.y), ptx::bf16hi(q.y));
  } else {
    const uint4 q = *(const uint4*)p;
    c.v[0] = make_float2(ptx::bf16lo(q.x), ptx::bf16hi(q.x));
    c.v[1] = make_float2(ptx::bf16lo(q.y), ptx::bf16hi(q.y));
    c.v[2] = make_float2(ptx::bf16lo(q.z), ptx::bf16hi(q.z));
    c.v[3] = make_float2(ptx::bf16lo(q.w), ptx::bf16hi(q.w));
  }
  return c;
}
template <int VEC, typename T>
__device__ __forceinline__ void store_ch(T* p, const Ch<VEC>& c) {
  if constexpr (VEC == 1) {
    *p = from_f<T>(c.v[0].x);
  } else if constexpr (VEC == 2 && sizeof(T) == 4) {
    *(float2*)p = c.v[0];
  } else if constexpr (VEC == 2) {
    *(uint32_t*)p = ptx::pack_bf16x2(c.v[0].x, c.v[0].y);
  } else if constexpr (sizeof(T) == 4) {
    *(float4*)p = make_float4(c.v[0].x, c.v[0].y, c.v[1].x, c.v[1].y);
  } else if constexpr (VEC == 4) {
    *(uint2*)p = make_uint2(ptx::pack_bf16x2(c.v[0].x, c.v[0].y),
                            ptx::pack_bf16x2(c.v[1].x, c.v[1].y));
  } else {
    *(uint4*)p = make_uint4(ptx::pack_bf16x2(c.v[0].x, c.v[0].y),
                            ptx::pack_bf16x2(c.v[1].x, c.v[1].y),
                            ptx::pack_bf16x2(c.v[2].x, c.v[2].y),
                            ptx::pack_bf16x2(c.v[3].x, c.v[3].y));
  }
}

// fp32 parameters of a thread's channels (NULL: all `other`).
template <int VEC>
__device__ __forceinline__ void load_param(float2 (&v)[kPairs(VEC)], const float* p, float other,
                                           bool al16) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) v[i] = make_float2(other, other);
  } else if (VEC >= 4 && al16) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 q = __ldg((const float4*)p + i);
      v[2 * i] = make_float2(q.x, q.y);
      v[2 * i + 1] = make_float2(q.z, q.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i)
      v[i] = make_float2(__ldg(p + 2 * i), VEC > 1 ? __ldg(p + 2 * i + 1) : other);
  }
}

// ---- slabs ----------------------------------------------------------------------
// A slab is one sample's frames of kk whole groups (W = kk C/G channels, at
// least 64 bytes of a frame where the groups allow).  A cluster of S blocks
// owns it, a contiguous share of its frames each.  The resident kernels
// (k_norm_*_res) copy their share into shared memory once and make every pass
// over it there, so that x (and dy) are read once from DRAM and y (dx) written
// once, which is the kernels' bound; slabs that a cluster cannot hold, and
// rows that are not 16-byte aligned, are read from global memory in every pass
// (k_norm_*_stream).
constexpr int NT = 128, NWARPS = NT / 32;
constexpr int MAX_KK = 128;
constexpr int MAX_S = 16;  // blocks in a cluster (8 where shares stay in global memory)
constexpr int SHARE = 64 * 1024;
constexpr int SMEM_MAX = SHARE + 32 * 1024;  // with room for sums (dynamic)

struct Slab {
  int kk, W, S;      // groups and channels per slab, blocks per slab
  int per_max;       // frames a block may own
  int slots;         // 16-byte vectors a thread of a resident kernel may own
  int cbv;           // vectors of a column block (all VEC-wide columns of W, at most NT)
  int pow2;          // cbv is a power of two <= 32: columns meet by shuffles first
  int nslabs;
  int uni;           // a thread's channels are of one group (and pow2): GroupSum applies
  int lanes;         // lane bits that share a group (uni)
  int two;           // a thread's channels are of two groups at most (not uni): TwoGroups
  int lg;            // log2 of the lanes that gather a group's sum (not uni)
  int keep;          // a block's slabs have the same channels
  int S_log, step_log;  // S; NT / cbv where cbv is a power of two
  FastDiv per_sample_div, cbv_div;
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
// A block's shared memory may be written by its cluster once it runs.  A kernel that
// writes to its peers says that it has started while its first loads are on their
// way, and waits for the others' word before its first write (the reading kernels
// meet a barrier ahead of their first read as it is).
template <int WRITES>
__device__ __forceinline__ void say_started(const Slab& sl) {
  if (WRITES && sl.S > 1) {
    __syncwarp();
    cluster_arrive();
  }
}
__device__ __forceinline__ void wait_started() {
  __syncwarp();
  cluster_wait();
}
// value at the same shared address of another block of the cluster
__device__ __forceinline__ float peer_f32(const float* p, int rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// write a value to the same shared address of another block of the cluster
__device__ __forceinline__ void to_peer_f32(float* p, int rank, float v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// Sums over the block's frames of NA quantities per channel, for the channels
// of the current column block: out(q, c, sum), c < n = cbv * VEC.  scr: NA * rows * n
// partial sums, rows the row groups of frames (warps, where columns meet by shuffles).
template <int NA, int VEC, typename F>
__device__ __forceinline__ void sum_channels(const Slab& sl, float2 (&acc)[NA][kPairs(VEC)],
                                             float* scr, int col, int rg, bool active, F out) {
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
  for (int c = threadIdx.x; c < NA * n; c += NT) {
    const int q = NA > 1 && c >= n;
    const float* d = scr + q * (rows - 1) * n + c;
    float t = 0.f;
#pragma unroll 8
    for (int r = 0; r < rows; ++r) t += d[r * n];
    out(q, c - q * n, t);
  }
  __syncthreads();
}
// The same into res[q * n + c], returned, behind the partial sums.
template <int NA, int VEC>
__device__ __forceinline__ const float* reduce_channels(const Slab& sl,
                                                        float2 (&acc)[NA][kPairs(VEC)],
                                                        float* scr, int col, int rg, bool active) {
  const int n = sl.cbv * VEC;
  float* res = scr + NA * n * (sl.pow2 ? NWARPS : NT / sl.cbv_div);
  sum_channels<NA, VEC>(sl, acc, scr, col, rg, active,
                        [&](int q, int c, float t) { res[q * n + c] = t; });
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

// gs[g] = the sum over the block of the values of group g's channels: v holds one
// per channel of the thread's column.  sl.lg lanes gather a group's values from
// the block's, so that all groups are summed at once.
template <int VEC>
__device__ __forceinline__ void gather_groups(const Slab& sl, int rows, int cg,
                                              const FastDiv& cg_div,
                                              const float2 (&v)[kPairs(VEC)], float* scr,
                                              float* gs) {
#pragma unroll
  for (int i = 0; i < kPairs(VEC); ++i) {
    scr[2 * i * NT + threadIdx.x] = v[i].x;
    scr[(2 * i + 1) * NT + threadIdx.x] = v[i].y;
  }
  __syncthreads();
  const int sub = threadIdx.x >> sl.lg, at = threadIdx.x & ((1 << sl.lg) - 1);
  const int n = min(rows, NT / sl.cbv_div) * cg;  // (row groups that hold frames)
  for (int g0 = 0; g0 < sl.kk; g0 += NT >> sl.lg) {  // (the same rounds for every thread)
    const int g = g0 + sub;
    float s = 0.f;
    if (g < sl.kk) {
      for (int k = at; k < n; k += 1 << sl.lg) {
        const int rg = k / cg_div, c = g * cg + k - rg * cg;
        s += scr[(c % VEC) * NT + rg * sl.cbv + c / VEC];
      }
    }
    for (int o = 1 << sl.lg >> 1; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (at == 0 && g < sl.kk) gs[g] = s;
  }
  __syncthreads();
}

// A thread's channels in two groups at most: those before `split` are of group
// g0, the others of g1.  A thread adds up its channels of either, and a group's
// lanes gather one value a thread and row of frames where gather_groups takes one
// for each channel.
template <int VEC>
struct TwoGroups {
  int g0, g1, split;
  __device__ __forceinline__ TwoGroups(const Slab& sl, int c, int cg, int g)
      : g0(g), g1(min(g + 1, sl.kk - 1)), split((g + 1) * cg - c) {}
  __device__ __forceinline__ float2 pick(int i, float lo, float hi) const {
    return make_float2(2 * i < split ? lo : hi, 2 * i + 1 < split ? lo : hi);
  }
  // (sum over g0's channels, sum over g1's)
  __device__ __forceinline__ float2 sums(const float2 (&v)[kPairs(VEC)]) const {
    float2 t = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) {
      t = __fadd2_rn(t, 2 * i < split ? make_float2(v[i].x, 0.f) : make_float2(0.f, v[i].x));
      t = __fadd2_rn(t, 2 * i + 1 < split ? make_float2(v[i].y, 0.f) : make_float2(0.f, v[i].y));
    }
    return t;
  }
};
// gs[q][g] = the sum over the block of v[q]'s parts of group g.
template <int VEC, int NQ>
__device__ __forceinline__ void gather_two(const Slab& sl, int rows, int cg,
                                           const float2 (&v)[NQ], float* scr,
                                           float* const (&gs)[NQ]) {
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    scr[2 * q * NT + threadIdx.x] = v[q].x;
    scr[(2 * q + 1) * NT + threadIdx.x] = v[q].y;
  }
  __syncthreads();
  const int sub = threadIdx.x >> sl.lg, at = threadIdx.x & ((1 << sl.lg) - 1);
  const int nr = min(rows, NT / sl.cbv_div);  // (row groups that hold frames)
  for (int g0 = 0; g0 < sl.kk; g0 += NT >> sl.lg) {  // (the same rounds for every thread)
    const int g = g0 + sub;
    float s[NQ] = {};
    if (g < sl.kk) {
      // columns v0 ... of the group; the first may be its owner's second group
      const int v0 = g * cg / VEC, nv = ((g + 1) * cg - 1) / VEC - v0 + 1;
      const int second = v0 * VEC < g * cg ? NT : 0;
      const uint32_t inv = 65536u / nv + 1;  // k / nv for k <= 2 NT
      for (int k = at; k < nr * nv; k += 1 << sl.lg) {
        const int r = (int)(k * inv >> 16), j = k - r * nv;
        const float* d = scr + r * sl.cbv + v0 + j + (j == 0 ? second : 0);
#pragma unroll
        for (int q = 0; q < NQ; ++q) s[q] += d[2 * q * NT];
      }
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      for (int o = 1 << sl.lg >> 1; o; o >>= 1) s[q] += __shfl_xor_sync(0xffffffffu, s[q], o);
      if (at == 0 && g < sl.kk) gs[q][g] = s[q];
    }
  }
  __syncthreads();
}

// Frames in flight per thread of the stream kernels, forward and backward: loads
// this narrow are bound by how many are under way (32 x 2000 x 1024 in one group:
// 141 us forward and 157 backward, with 4 and 2 frames 164 and 208; 333 channels,
// an element a thread: 286 and 351, with 4 and 2 frames 350 and 665).
template <int VEC>
constexpr int kFlyFwd = VEC <= 2 ? 16 : 8;
template <int VEC>
constexpr int kFlyBwd = VEC <= 2 ? 8 : 4;

// The block's slab, frames and column.
template <int VEC>
struct Where {
  int b, c0, rank, tb, t0, rows, v, rg, step;
  bool active;
};
template <int VEC>
__device__ __forceinline__ void set_frames(Where<VEC>& w, const NormArgs& a, const Slab& sl,
                                           int length) {
  w.tb = frames_of(a, length);
  const int per = (w.tb + sl.S - 1) >> sl.S_log;
  w.t0 = min(w.tb, w.rank * per);
  w.rows = min(w.tb, w.t0 + per) - w.t0;
}
template <int VEC>
__device__ __forceinline__ Where<VEC> where(const NormArgs& a, const Slab& sl, int slab, int rank,
                                            int length) {
  Where<VEC> w;
  w.rank = rank;
  w.b = slab / sl.per_sample_div;
  w.c0 = (slab - w.b * (int)sl.per_sample_div.d) * sl.W;
  w.rg = (int)threadIdx.x / sl.cbv_div;
  w.v = threadIdx.x - w.rg * sl.cbv;
  w.step = NT / sl.cbv_div;
  w.active = w.rg < w.step;
  set_frames(w, a, sl, length);
  return w;
}

// zeros in the block's share of the frames past the sample's length
template <int VEC, typename T>
__device__ __forceinline__ void zero_tail(const NormArgs& a, const Slab& sl, const Where<VEC>& w,
                                          T* out, long long ld) {
  const int left = a.T - w.tb, per = (left + sl.S - 1) >> sl.S_log;
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
__device__ __forceinline__ int rows_of(const Where<VEC>& w, const Slab& sl) {
  if (!w.active || w.rg >= w.rows) return 0;
  const int last = w.rows - 1 - w.rg;
  return (sl.pow2 ? last >> sl.step_log : last / w.step) + 1;
}

// The blocks' (n, mean, M2) of a slab, joined in order; st: the cluster's
// [group] (mean, M2) and n at the same shared addresses of every block.
__device__ __forceinline__ void join_stats(const NormArgs& a, const Slab& sl, int b, int c0,
                                           int rank, const float* mean_s, const float* m2_s,
                                           const float* n_s, float* mean_t, float* rstd_t) {
  for (int g = threadIdx.x; g < sl.kk; g += NT) {
    float nt = 0.f, mt = 0.f, st = 0.f;
    for (int k = 0; k < sl.S; ++k) {
      const float nk = sl.S > 1 ? peer_f32(n_s, k) : *n_s;
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
    if (rank == 0) a.stats[(long long)b * a.G + c0 / a.cg_div + g] = make_float2(mt, rstd);
  }
}

// Sums and squares of a thread's frames of its channels about the first of
// them (its few frames lose no digits to that, wherever the mean is), then the
// thread's mean and its squares about that: q - s^2 / k.
template <int VEC>
struct Partial {
  float2 first[kPairs(VEC)], s[kPairs(VEC)], q[kPairs(VEC)];
  __device__ __forceinline__ void begin(const Ch<VEC>& c) {
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) {
      first[i] = make_float2(-c.v[i].x, -c.v[i].y);
      s[i] = q[i] = make_float2(0.f, 0.f);
    }
  }
  __device__ __forceinline__ void add(const Ch<VEC>& c) {
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) {
      const float2 d = __fadd2_rn(c.v[i], first[i]);
      s[i] = __fadd2_rn(s[i], d);
      q[i] = __ffma2_rn(d, d, q[i]);
    }
  }
  // s: the thread's mean, q: squares about it
  __device__ __forceinline__ void end(int cnt) {
    const float rk = __frcp_rn((float)cnt);
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) {
      const float2 mk = __fmul2_rn(s[i], make_float2(rk, rk));
      q[i] = __ffma2_rn(make_float2(-s[i].x, -s[i].y), mk, q[i]);
      s[i] = __fadd2_rn(mk, make_float2(-first[i].x, -first[i].y));
    }
  }
  // the same for a thread of two groups at most, of means (lo, hi)
  __device__ __forceinline__ float2 out(const TwoGroups<VEC>& tw, int half, int cnt, float lo,
                                        float hi) const {
    const float k = (float)cnt;
    float2 v[kPairs(VEC)];
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) {
      const float2 mean = tw.pick(i, lo, hi);
      const float2 d = __fadd2_rn(s[i], make_float2(-mean.x, -mean.y));
      v[i] = half == 0 ? __fmul2_rn(make_float2(k, k), s[i])
                       : __ffma2_rn(__fmul2_rn(d, d), make_float2(k, k), q[i]);
    }
    return tw.sums(v);
  }
  // half 0: the sum; half 1: the squares about the groups' means
  __device__ __forceinline__ void out(float2 (&acc)[1][kPairs(VEC)], int half, int cnt, int c,
                                      const float* mean_s, const FastDiv& cg) const {
    const float2 k = make_float2((float)cnt, (float)cnt);
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) {
      if (half == 0) {
        acc[0][i] = __fmul2_rn(k, s[i]);
      } else {
        const int ca = c + 2 * i, cz = VEC > 1 ? ca + 1 : ca;
        const float2 d = __fadd2_rn(s[i], make_float2(-mean_s[ca / cg], -mean_s[cz / cg]));
        acc[0][i] = __ffma2_rn(__fmul2_rn(d, d), k, q[i]);
      }
    }
  }
};

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(NT, 5)
k_norm_fwd_stream(NormArgs a, Slab sl, const T* __restrict__ x, T* __restrict__ y) {
  extern __shared__ __align__(16) unsigned char smem[];
  // (mean_s, m2_s and n_s are read by the cluster's other blocks)
  __shared__ float gs[2][MAX_KK], mean_cb[MAX_KK], mean_s[MAX_KK], m2_s[MAX_KK], n_s;
  __shared__ float mean_t[MAX_KK], rstd_t[MAX_KK];
  float* scr = (float*)smem;
  const int slab = (int)blockIdx.x >> sl.S_log;
  const Where<VEC> w = where<VEC>(a, sl, slab, blockIdx.x - slab * sl.S,
                                  length_of(a, slab / sl.per_sample_div));
  const T* src = x + w.b * a.xb + w.c0 + (long long)w.t0 * a.xf;
  T* ys = y + w.b * a.yb + w.c0;
  zero_tail<VEC, T>(a, sl, w, ys, a.yf);
  const long long ld = a.xf, inc = ld * w.step;
  const int nb = sl.cbv * VEC, cnt = rows_of(w, sl);
  for (int g = threadIdx.x; g < sl.kk; g += NT) gs[0][g] = gs[1][g] = mean_s[g] = m2_s[g] = 0.f;
  if (threadIdx.x == 0) n_s = (float)w.rows * a.cg;
  __syncthreads();
#pragma unroll 1
  for (int cb = 0; cb < sl.W; cb += nb) {
    const int c = cb + w.v * VEC;
    const bool in = w.active && c < sl.W;
    Partial<VEC> st;
    if (in && cnt > 0) {
      const T* p = src + w.rg * ld + c;
      st.begin(load_ch<VEC, T>(p));
#pragma unroll (kFlyFwd<VEC>)
      for (int k = 0; k < cnt; ++k, p += inc) st.add(load_ch<VEC, T>(p));
      st.end(cnt);
    }
    // the column block's sums, then its squares about its own means
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      float2 acc[1][kPairs(VEC)] = {};
      if (in && cnt > 0) st.out(acc, half, cnt, c, mean_cb, a.cg_div);
      const float* res = reduce_channels<1, VEC>(sl, acc, scr, w.v, w.rg, in);
      reduce_groups<1, VEC>(sl, a.cg, cb, res, gs + half, [](int) { return 1.f; });
      __syncthreads();
      for (int g = threadIdx.x; g < sl.kk; g += NT) {
        // the group's channels in this column block, and in those before
        const int g0 = g * a.cg, now = min(g0 + a.cg, min(cb + nb, sl.W)) - max(g0, cb);
        if (now <= 0 || w.rows == 0) continue;
        const float n1 = (float)w.rows * now, n0 = (float)w.rows * max(0, cb - g0);
        if (half == 0) {
          mean_cb[g] = gs[0][g] / n1;
          gs[0][g] = 0.f;
        } else {
          const float d = mean_cb[g] - mean_s[g], f = n1 / (n0 + n1);
          mean_s[g] += d * f;
          m2_s[g] += gs[1][g] + d * d * (n0 * f);
          gs[1][g] = 0.f;
        }
      }
      __syncthreads();
    }
  }
  if (sl.S > 1) {
    cluster_arrive();
    cluster_wait();
  }
  join_stats(a, sl, w.b, w.c0, w.rank, mean_s, m2_s, &n_s, mean_t, rstd_t);
  __syncthreads();
  if (sl.S > 1) cluster_arrive();  // (waited for at the end: peers may still read)
  T* yt = ys + (long long)w.t0 * a.yf;
#pragma unroll 1
  for (int cb = 0; cb < sl.W; cb += nb) {
    const int c = cb + w.v * VEC;
    if (cnt == 0 || c >= sl.W) continue;
    float2 m[kPairs(VEC)], s[kPairs(VEC)], be[kPairs(VEC)];
    load_param<VEC>(s, a.gamma ? a.gamma + w.c0 + c : nullptr, 1.f, false);
    load_param<VEC>(be, a.beta ? a.beta + w.c0 + c : nullptr, 0.f, false);
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) {
      const int ca = c + 2 * i, cz = VEC > 1 ? ca + 1 : ca;
      const int gx = ca / a.cg_div, gz = cz / a.cg_div;
      m[i] = make_float2(-mean_t[gx], -mean_t[gz]);
      s[i] = __fmul2_rn(make_float2(rstd_t[gx], rstd_t[gz]), s[i]);
    }
    const T* p = src + w.rg * ld + c;
    T* o = yt + w.rg * a.yf + c;
    const long long oinc = w.step * a.yf;
#pragma unroll (kFlyFwd<VEC>)
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

// The backward's two uses of a frame, in d = x - mean and s = rstd gamma:
//   u = s d + beta,  g = dy act'(u),  sums of g d and g (rstd goes onto the sums),
//   dx = s g + (k1 + k2 d),  k1 = -rstd m1,  k2 = -rstd^2 m2.
// Both uses take sigmoid2 in bf16 too: the unit's tanh, one operation where that has
// two, is 5% faster (1024 x 1000 x 512: 485 us against 509), but its error of 2^-11 of
// tanh(u / 2) moves act' by up to 2^-12 |t| |1 - u t|, whatever act' itself is: at u = -8
// 1.7e-3 of an act' of -2.3e-3.
template <typename T, int VEC, int ACT>
struct Back {
  float2 m[kPairs(VEC)], rs[kPairs(VEC)], ga[kPairs(VEC)], be[kPairs(VEC)];
  __device__ __forceinline__ void stats(const float2* st, int c, const FastDiv& cg) {
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) {
      const int ca = c + 2 * i, cz = VEC > 1 ? ca + 1 : ca;
      const float2 p = st[ca / cg], q = st[cz / cg];
      m[i] = make_float2(-p.x, -q.x);
      rs[i] = make_float2(p.y, q.y);
    }
  }
  struct Sums {
    float2 m[kPairs(VEC)], s[kPairs(VEC)], be[kPairs(VEC)];
    __device__ __forceinline__ void add(const Ch<VEC>& x, const Ch<VEC>& dy,
                                        float2 (&acc)[2][kPairs(VEC)]) const {
#pragma unroll
      for (int i = 0; i < kPairs(VEC); ++i) {
        const float2 d = __fadd2_rn(x.v[i], m[i]);
        const float2 g = dact2<ACT, T>(dy.v[i], __ffma2_rn(d, s[i], be[i]));
        acc[0][i] = __ffma2_rn(g, d, acc[0][i]);
        acc[1][i] = __fadd2_rn(acc[1][i], g);
      }
    }
  };
  struct Dx {
    float2 m[kPairs(VEC)], s[kPairs(VEC)], be[kPairs(VEC)], k1[kPairs(VEC)], k2[kPairs(VEC)];
    __device__ __forceinline__ Ch<VEC> of(const Ch<VEC>& x, const Ch<VEC>& dy) const {
      Ch<VEC> o;
#pragma unroll
      for (int i = 0; i < kPairs(VEC); ++i) {
        const float2 d = __fadd2_rn(x.v[i], m[i]), u = __ffma2_rn(d, s[i], be[i]);
        const float2 k = __ffma2_rn(d, k2[i], k1[i]);
        o.v[i] = __ffma2_rn(dact2<ACT, T>(dy.v[i], u), s[i], k);
      }
      return o;
    }
  };
  __device__ __forceinline__ Sums sums() const {
    Sums q;
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) {
      q.m[i] = m[i];
      q.s[i] = __fmul2_rn(rs[i], ga[i]);
      q.be[i] = be[i];
    }
    return q;
  }
  // g (x - mean) to g xh
  __device__ __forceinline__ void scale(float2 (&acc)[kPairs(VEC)]) const {
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) acc[i] = __fmul2_rn(acc[i], rs[i]);
  }
  // k1, k2: minus the means of gamma g and gamma g xh.  A group of one value (one)
  // passes no gradient on, where the three terms would cancel but for their rounding.
  __device__ __forceinline__ Dx dx(const float2 (&k1)[kPairs(VEC)],
                                   const float2 (&k2)[kPairs(VEC)], bool one) const {
    Dx q;
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) {
      q.m[i] = m[i];
      const float2 r = one ? make_float2(0.f, 0.f) : rs[i];
      q.s[i] = __fmul2_rn(r, ga[i]);
      q.be[i] = be[i];
      q.k1[i] = __fmul2_rn(r, k1[i]);
      q.k2[i] = __fmul2_rn(__fmul2_rn(r, r), k2[i]);
    }
    return q;
  }
};

// Minus the means of gamma g and gamma g xh for a thread's channels.
template <int VEC>
__device__ __forceinline__ void means_of(const float* m1_t, const float* m2_t, int c,
                                         const FastDiv& cg, float2 (&k1)[kPairs(VEC)],
                                         float2 (&k2)[kPairs(VEC)]) {
#pragma unroll
  for (int i = 0; i < kPairs(VEC); ++i) {
    const int ca = c + 2 * i, gx = ca / cg, gz = (VEC > 1 ? ca + 1 : ca) / cg;
    k1[i] = make_float2(-m1_t[gx], -m1_t[gz]);
    k2[i] = make_float2(-m2_t[gx], -m2_t[gz]);
  }
}

// m1, m2 of the slab's groups from the blocks' sums gs2 and gs1, in order.
__device__ __forceinline__ void join_means(const NormArgs& a, const Slab& sl, int tb,
                                           const float* gs2, const float* gs1, float* m1_t,
                                           float* m2_t) {
  const float n = (float)tb * a.cg;
  for (int g = threadIdx.x; g < sl.kk; g += NT) {
    float s2 = 0.f, s1 = 0.f;
    for (int k = 0; k < sl.S; ++k) {
      s2 += sl.S > 1 ? peer_f32(gs2 + g, k) : gs2[g];
      s1 += sl.S > 1 ? peer_f32(gs1 + g, k) : gs1[g];
    }
    m1_t[g] = n > 0.f ? s1 / n : 0.f;
    m2_t[g] = n > 0.f ? s2 / n : 0.f;
  }
}

// part: per slab block and channel (sum g xh, sum g), [B][S][C].
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(NT, 5)
k_norm_bwd_stream(NormArgs a, Slab sl, const T* __restrict__ x, const T* __restrict__ dy,
                  T* __restrict__ dx, float2* __restrict__ part) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float gs[2][MAX_KK];  // read by the cluster's other blocks
  __shared__ float m1_t[MAX_KK], m2_t[MAX_KK];
  float* scr = (float*)smem;
  const int slab = (int)blockIdx.x >> sl.S_log;
  const Where<VEC> w = where<VEC>(a, sl, slab, blockIdx.x - slab * sl.S,
                                  length_of(a, slab / sl.per_sample_div));
  const T* xs = x + w.b * a.xb + w.c0 + (long long)w.t0 * a.xf;
  const T* ds = dy + w.b * a.yb + w.c0 + (long long)w.t0 * a.yf;
  T* os = dx + w.b * a.xb + w.c0;
  zero_tail<VEC, T>(a, sl, w, os, a.xf);
  os += (long long)w.t0 * a.xf;
  const long long xinc = a.xf * w.step, dinc = a.yf * w.step;
  const int nb = sl.cbv * VEC, cnt = rows_of(w, sl);
  const float2* stats = a.stats + (long long)w.b * a.G + w.c0 / a.cg_div;
  for (int g = threadIdx.x; g < sl.kk; g += NT) gs[0][g] = gs[1][g] = 0.f;
  __syncthreads();
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int cb = 0; cb < sl.W; cb += nb) {
      const int c = cb + w.v * VEC;
      const bool in = w.active && c < sl.W;
      Back<T, VEC, ACT> bk;
      if (in) {
        bk.stats(stats, c, a.cg_div);
        load_param<VEC>(bk.ga, a.gamma ? a.gamma + w.c0 + c : nullptr, 1.f, false);
        load_param<VEC>(bk.be, a.beta ? a.beta + w.c0 + c : nullptr, 0.f, false);
      }
      const T *px = xs + w.rg * a.xf + c, *pd = ds + w.rg * a.yf + c;
      if (pass == 0) {
        float2 acc[2][kPairs(VEC)] = {};
        if (in) {
          const auto sums = bk.sums();
#pragma unroll (kFlyBwd<VEC>)
          for (int k = 0; k < cnt; ++k, px += xinc, pd += dinc)
            sums.add(load_ch<VEC, T>(px), load_ch<VEC, T>(pd), acc);
          bk.scale(acc[0]);
        }
        const float* res = reduce_channels<2, VEC>(sl, acc, scr, w.v, w.rg, in);
        for (int k = threadIdx.x; k < nb && cb + k < sl.W; k += NT)
          part[((long long)w.b * sl.S + w.rank) * a.C + w.c0 + cb + k] =
              make_float2(res[k], res[nb + k]);
        reduce_groups<2, VEC>(sl, a.cg, cb, res, gs, [&](int ch) {
          return a.gamma ? a.gamma[w.c0 + ch] : 1.f;
        });
      } else if (in) {
        float2 k1[kPairs(VEC)], k2[kPairs(VEC)];
        means_of<VEC>(m1_t, m2_t, c, a.cg_div, k1, k2);
        const auto last = bk.dx(k1, k2, w.tb == 1 && a.cg == 1);
        T* po = os + w.rg * a.xf + c;
#pragma unroll (kFlyBwd<VEC>)
        for (int k = 0; k < cnt; ++k, px += xinc, pd += dinc, po += xinc)
          store_ch<VEC, T>(po, last.of(load_ch<VEC, T>(px), load_ch<VEC, T>(pd)));
      }
    }
    if (pass) break;
    __syncthreads();
    if (sl.S > 1) {
      cluster_arrive();
      cluster_wait();
    }
    join_means(a, sl, w.tb, gs[0], gs[1], m1_t, m2_t);
    __syncthreads();
    if (sl.S > 1) cluster_arrive();  // (waited for at the end: peers may still read)
  }
  __syncwarp();
  if (sl.S > 1) cluster_wait();
}

// Sum of one value per thread over the block's threads of the same group, for
// slabs whose threads hold channels of one group each: shuffles over the lane
// bits in sl.lanes, then the warps' sums from buf[group][warp] in order.
__device__ __forceinline__ float group_lanes(float v, int lanes) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    if (lanes & o) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float group_warps(const float (*buf)[NWARPS], int g) {
  static_assert(NWARPS == 4, "one 16-byte read");
  const float4 q = *(const float4*)buf[g];
  return ((q.x + q.y) + q.z) + q.w;
}

// ---- resident kernels -------------------------------------------------------------
// A block walks slabs.  A thread owns one 16-byte column of its block's share,
// every step-th frame, and is the only reader of its shared-memory slots: it
// waits for its own copies alone, and as soon as the last pass has read a slot
// it copies the next slab's frame into it.  So the loads of the next slab run
// under the last pass of this one, with no barrier between them, and the blocks
// of an SM (three at the 64 KB share) overlap one's reductions with another's
// passes.
template <typename T>
constexpr int kVec16 = 16 / (int)sizeof(T);

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int SLOT = NT * 16;  // bytes from one of a thread's slots to its next

// The last pass over `cnt` slots, with the next slab's `ncnt` frames copied into
// the slots behind it, in two copy groups.  Returns the slots of the first.
// (Two frames at a time: the copies order memory, so a frame's loads would not
// start before the one ahead has stored.)
template <typename A, typename F>
__device__ __forceinline__ int turn_over(int cnt, int ncnt, A apply, F fetch) {
  using Two = std::integral_constant<int, 2>;
  using One = std::integral_constant<int, 1>;
  const int both = min(cnt, ncnt) & ~1, head = (both / 2) & ~1;
  int k = 0;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int end = part ? both : head;
#pragma unroll 1
    for (; k < end; k += 2) {
      apply(k, Two{});
      fetch(k);
      fetch(k + 1);
    }
    if (part == 0) copy_commit();
  }
  // what only one of the two slabs has; a frame is copied in once its slot is read
  const int done = k;
#pragma unroll 1
  for (; k + 2 <= cnt; k += 2) apply(k, Two{});
  if (k < cnt) apply(k, One{});
  for (k = done; k < ncnt; ++k) fetch(k);
  copy_commit();
  return head;
}

// The block's next slab: the same channels of a later sample (keep), or any.
template <int VEC>
__device__ __forceinline__ void next_where(Where<VEC>& w, const NormArgs& a, const Slab& sl,
                                           int slab, int stride, int length) {
  if (sl.keep) {
    w.b += stride / sl.per_sample_div;
    set_frames(w, a, sl, length);
  } else {
    w = where<VEC>(a, sl, slab, w.rank, length);
  }
}

// Length of the block's slab after next, asked for one slab ahead of its use.
__device__ __forceinline__ int length_ahead(const NormArgs& a, const Slab& sl, int slab) {
  return slab < sl.nslabs ? length_of(a, slab / sl.per_sample_div) : 0;
}

template <typename T, int ACT, int UNI>
__global__ void __launch_bounds__(NT, 3)
k_norm_fwd_res(NormArgs a, Slab sl, const T* __restrict__ x, T* __restrict__ y) {
  constexpr int VEC = kVec16<T>, NP = kPairs(VEC);
  extern __shared__ __align__(16) unsigned char smem[];
  // (what other blocks of the cluster read or write has a set per parity of the
  // slab count, so that one barrier a slab keeps writers off what is still read)
  constexpr int GK = UNI ? 1 : MAX_KK, UK = UNI ? 32 : 1;
  __shared__ float mean_s[2][GK], m2_s[2][GK], n_s[2];
  __shared__ float mean_t[GK], rstd_t[GK];
  __shared__ __align__(16) float buf[2][UK][NWARPS];
  // (mean, M2) of every block of the cluster (UNI): [parity][block][2][group]
  float* from = (float*)(smem + (size_t)sl.slots * SLOT);
  float* scr = from;
  const unsigned char* mine = smem + threadIdx.x * 16;
  const uint32_t mine_a = ptx::smem_u32(mine);
  const int first = (int)blockIdx.x >> sl.S_log, rank = blockIdx.x - first * sl.S;
  const int stride = (int)gridDim.x >> sl.S_log, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool al16 = (((uintptr_t)a.gamma | (uintptr_t)a.beta) & 15) == 0;
  Where<VEC> w = where<VEC>(a, sl, first, rank, length_of(a, first / sl.per_sample_div));
  int ahead = length_ahead(a, sl, first + stride);
  const int c = w.v * VEC, myg = c / a.cg_div;
  const TwoGroups<VEC> tw(sl, c, a.cg, myg);
  int cnt = rows_of(w, sl);
  const long long xinc = a.xf * w.step, yinc = a.yf * w.step;
  {
    const T* p = x + w.b * a.xb + w.c0 + (long long)(w.t0 + w.rg) * a.xf + c;
    for (int k = 0; k < cnt; ++k, p += xinc) copy16(mine_a + k * SLOT, p);
    copy_commit();
    copy_commit();
  }
  say_started<UNI>(sl);
  int ready = cnt;  // slots of the first of the two copy groups
  int par = 0;
  float2 ga[NP], be[NP];
#pragma unroll 1
  for (int slab = first; slab < sl.nslabs; slab += stride, par ^= 1) {
    const bool more = slab + stride < sl.nslabs;
    Where<VEC> nx = w;
    int ncnt = 0;
    if (more) {
      next_where(nx, a, sl, slab + stride, stride, ahead);
      ncnt = rows_of(nx, sl);
    }
    ahead = length_ahead(a, sl, slab + 2 * stride);
    T* ys = y + w.b * a.yb + w.c0;
    if (w.active && (!sl.keep || slab == first)) {
      load_param<VEC>(ga, a.gamma ? a.gamma + w.c0 + c : nullptr, 1.f, al16);
      load_param<VEC>(be, a.beta ? a.beta + w.c0 + c : nullptr, 0.f, al16);
    }
    zero_tail<VEC, T>(a, sl, w, ys, a.yf);
    const float n = (float)w.rows * a.cg;
    float2 s[NP], m[NP];
    Partial<VEC> st;
    copy_wait<1>();
    if (cnt > 0) {
      if (ready == 0) copy_wait<0>();
      st.begin(load_ch<VEC, T>((const T*)mine));
#pragma unroll 4
      for (int k = 0; k < ready; ++k) st.add(load_ch<VEC, T>((const T*)(mine + k * SLOT)));
      copy_wait<0>();
#pragma unroll 4
      for (int k = ready; k < cnt; ++k) st.add(load_ch<VEC, T>((const T*)(mine + k * SLOT)));
      st.end(cnt);
    }
    if constexpr (UNI) {
      // the thread's (count, mean, squares about it) over its channels; then
      // the block's mean, then the squares about that
      float tn = 0.f, tm = 0.f, tq = 0.f;
      if (cnt > 0) {
        float2 ms = st.s[0], qs = st.q[0];
#pragma unroll
        for (int i = 1; i < NP; ++i) {
          ms = __fadd2_rn(ms, st.s[i]);
          qs = __fadd2_rn(qs, st.q[i]);
        }
        tm = (ms.x + ms.y) * (1.f / VEC);
        float2 ds = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const float2 d = __fadd2_rn(st.s[i], make_float2(-tm, -tm));
          ds = __ffma2_rn(d, d, ds);
        }
        tq = fmaf(ds.x + ds.y, (float)cnt, qs.x + qs.y);
        tn = (float)(cnt * VEC);
      }
      const float rn = __frcp_rn(fmaxf(n, 1.f));
      const bool leader = (lane & sl.lanes) == 0;
      float v = group_lanes(tn * tm, sl.lanes);
      if (leader) buf[0][myg][warp] = v;
      __syncthreads();
      float mean = group_warps(buf[0], myg) * rn;
      const float d = tm - mean;
      v = group_lanes(fmaf(tn * d, d, tq), sl.lanes);
      if (leader) buf[1][myg][warp] = v;
      __syncthreads();
      float m2 = group_warps(buf[1], myg), all = n;
      if (sl.S > 1) {
        if (slab == first) wait_started();
        if (leader && warp == 0)
          for (int k = 0; k < sl.S; ++k) {
            to_peer_f32(from + (par * sl.S + rank) * 2 * sl.kk + myg, k, mean);
            to_peer_f32(from + ((par * sl.S + rank) * 2 + 1) * sl.kk + myg, k, m2);
          }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        const int per = (w.tb + sl.S - 1) >> sl.S_log;  // frames of the blocks but the last
        float mt = 0.f, sq = 0.f;
        all = 0.f;
        for (int k = 0; k < sl.S; ++k) {
          const float nk = (float)(min(w.tb, (k + 1) * per) - min(w.tb, k * per)) * a.cg;
          const float* fk = from + (par * sl.S + k) * 2 * sl.kk + myg;
          const float mk = fk[0], sk = fk[sl.kk];
          if (nk == 0.f) break;
          // (an approximate quotient and root, 2 units in the last place, once a group)
          const float dk = mk - mt, f = __fdividef(nk, all + nk);
          mt = fmaf(dk, f, mt);
          sq += fmaf(dk * dk, all * f, sk);
          all += nk;
        }
        mean = mt;
        m2 = sq;
      }
      const float rstd =
          all > 0.f ? rsqrtf(fmaf(m2, __frcp_rn(fmaxf(all, 1.f)), a.eps)) : 0.f;
      if (rank == 0 && warp == 0 && leader)
        a.stats[(long long)w.b * a.G + w.c0 / a.cg_div + myg] =
            make_float2(all > 0.f ? mean : 0.f, rstd);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        m[i] = make_float2(-mean, -mean);
        s[i] = __fmul2_rn(make_float2(rstd, rstd), ga[i]);
      }
    } else {
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        float* to = half ? m2_s[par] : mean_s[par];
        if (sl.two) {
          float2 v[1] = {make_float2(0.f, 0.f)};
          if (cnt > 0)
            v[0] = st.out(tw, half, cnt, half ? mean_s[par][tw.g0] : 0.f,
                          half ? mean_s[par][tw.g1] : 0.f);
          gather_two<VEC, 1>(sl, w.rows, a.cg, v, scr, {to});
        } else {
          float2 acc[1][NP] = {};
          if (cnt > 0) st.out(acc, half, cnt, c, mean_s[par], a.cg_div);
          gather_groups<VEC>(sl, w.rows, a.cg, a.cg_div, acc[0], scr, to);
        }
        if (half == 0) {
          for (int g = threadIdx.x; g < sl.kk; g += NT)
            mean_s[par][g] = w.rows ? mean_s[par][g] / n : 0.f;
          if (threadIdx.x == 0) n_s[par] = n;
          __syncthreads();
        }
      }
      if (sl.S > 1) {
        cluster_arrive();
        cluster_wait();
      }
      join_stats(a, sl, w.b, w.c0, rank, mean_s[par], m2_s[par], &n_s[par], mean_t, rstd_t);
      __syncthreads();
      if (w.active && sl.two) {
        const float ml = mean_t[tw.g0], mh = mean_t[tw.g1];
        const float rl = rstd_t[tw.g0], rh = rstd_t[tw.g1];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          m[i] = tw.pick(i, -ml, -mh);
          s[i] = __fmul2_rn(tw.pick(i, rl, rh), ga[i]);
        }
      } else if (w.active) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int ca = c + 2 * i, gx = ca / a.cg_div, gz = (ca + 1) / a.cg_div;
          m[i] = make_float2(-mean_t[gx], -mean_t[gz]);
          s[i] = __fmul2_rn(make_float2(rstd_t[gx], rstd_t[gz]), ga[i]);
        }
      }
    }
    // last pass: write y, copy the next slab into the slots it has read
    T* o = ys + (long long)(w.t0 + w.rg) * a.yf + c;
    const T* p = x + nx.b * a.xb + nx.c0 + (long long)(nx.t0 + nx.rg) * a.xf + c;
    auto apply = [&](int k, auto frames) {
      constexpr int U = decltype(frames)::value;
      Ch<VEC> q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) q[u] = load_ch<VEC, T>((const T*)(mine + (k + u) * SLOT));
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
          q[u].v[i] = act2<ACT, T>(__ffma2_rn(__fadd2_rn(q[u].v[i], m[i]), s[i], be[i]));
        store_ch<VEC, T>(o, q[u]);
        o += yinc;
      }
    };
    auto fetch = [&](int k) {
      copy16(mine_a + k * SLOT, p);
      p += xinc;
    };
    ready = turn_over(cnt, ncnt, apply, fetch);
    w = nx;
    cnt = ncnt;
  }
  __syncwarp();
  if (sl.S > 1) {  // peers may still read this block's statistics
    cluster_arrive();
    cluster_wait();
  }
}

// part: sums per block (keep) or per sample, block and channel of (g xh, g).
template <typename T, int ACT, int UNI>
__global__ void __launch_bounds__(NT, 3)
k_norm_bwd_res(NormArgs a, Slab sl, const T* __restrict__ x, const T* __restrict__ dy,
               T* __restrict__ dx, float2* __restrict__ part) {
  constexpr int VEC = kVec16<T>, NP = kPairs(VEC);
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int GK = UNI ? 1 : MAX_KK, UK = UNI ? 32 : 1;
  __shared__ float gs[2][2][UNI ? 1 : MAX_KK];  // by parity; read by the cluster's other blocks
  __shared__ float m1_t[GK], m2_t[GK];
  __shared__ __align__(16) float buf[2][2][UK][NWARPS];
  const int half_bytes = sl.slots * SLOT;
  // sums of every block of the cluster (UNI): [parity][block][2][group]
  float* from = (float*)(smem + 2 * (size_t)half_bytes);
  float* scr = from + (UNI ? 4 * sl.S * sl.kk : 0);
  const unsigned char* mine = smem + threadIdx.x * 16;
  const uint32_t mine_a = ptx::smem_u32(mine);
  const int first = (int)blockIdx.x >> sl.S_log, rank = blockIdx.x - first * sl.S;
  const int stride = (int)gridDim.x >> sl.S_log, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool al16 = (((uintptr_t)a.gamma | (uintptr_t)a.beta) & 15) == 0;
  Where<VEC> w = where<VEC>(a, sl, first, rank, length_of(a, first / sl.per_sample_div));
  int ahead = length_ahead(a, sl, first + stride);
  const int c = w.v * VEC, myg = c / a.cg_div;
  const TwoGroups<VEC> tw(sl, c, a.cg, myg);
  int cnt = rows_of(w, sl);
  const long long xinc = a.xf * w.step, dinc = a.yf * w.step;
  {
    const T* p = x + w.b * a.xb + w.c0 + (long long)(w.t0 + w.rg) * a.xf + c;
    const T* d = dy + w.b * a.yb + w.c0 + (long long)(w.t0 + w.rg) * a.yf + c;
    for (int k = 0; k < cnt; ++k, p += xinc, d += dinc) {
      copy16(mine_a + k * SLOT, p);
      copy16(mine_a + half_bytes + k * SLOT, d);
    }
    copy_commit();
    copy_commit();
  }
  say_started<UNI>(sl);
  int ready = cnt, par = 0;
  Back<T, VEC, ACT> bk;
  // (a slab's statistics are asked for one slab ahead)
  auto stats_of = [&](const Where<VEC>& q) {
    return a.stats[(long long)q.b * a.G + q.c0 / a.cg_div + myg];
  };
  float2 stat = UNI ? stats_of(w) : make_float2(0.f, 0.f);
  float2 tot[2][NP] = {};  // sums of all the block's slabs with these channels
#pragma unroll 1
  for (int slab = first; slab < sl.nslabs; slab += stride, par ^= 1) {
    const bool more = slab + stride < sl.nslabs;
    T* os = dx + w.b * a.xb + w.c0;
    if constexpr (UNI) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        bk.m[i] = make_float2(-stat.x, -stat.x);
        bk.rs[i] = make_float2(stat.y, stat.y);
      }
    } else if (w.active) {
      const float2* st = a.stats + (long long)w.b * a.G + w.c0 / a.cg_div;
      if (sl.two) {
        const float2 lo = st[tw.g0], hi = st[tw.g1];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          bk.m[i] = tw.pick(i, -lo.x, -hi.x);
          bk.rs[i] = tw.pick(i, lo.y, hi.y);
        }
      } else {
        bk.stats(st, c, a.cg_div);
      }
    }
    if (w.active && (!sl.keep || slab == first)) {
      load_param<VEC>(bk.ga, a.gamma ? a.gamma + w.c0 + c : nullptr, 1.f, al16);
      load_param<VEC>(bk.be, a.beta ? a.beta + w.c0 + c : nullptr, 0.f, al16);
    }
    float2 acc[2][NP] = {};
    // the next slab, and the zeros past this one's frames: work for the time
    // that the blocks of a cluster wait for one another
    Where<VEC> nx = w;
    int ncnt = 0;
    auto meanwhile = [&]() {
      if (more) {
        next_where(nx, a, sl, slab + stride, stride, ahead);
        ncnt = rows_of(nx, sl);
        if (UNI) stat = stats_of(nx);
      }
      ahead = length_ahead(a, sl, slab + 2 * stride);
      zero_tail<VEC, T>(a, sl, w, os, a.xf);
    };
    const auto pass = bk.sums();
    auto sums = [&](int k) {
      pass.add(load_ch<VEC, T>((const T*)(mine + k * SLOT)),
               load_ch<VEC, T>((const T*)(mine + half_bytes + k * SLOT)), acc);
    };
    copy_wait<1>();
#pragma unroll 2
    for (int k = 0; k < ready; ++k) sums(k);
    copy_wait<0>();
#pragma unroll 2
    for (int k = ready; k < cnt; ++k) sums(k);
    bk.scale(acc[0]);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      tot[0][i] = __fadd2_rn(tot[0][i], acc[0][i]);
      tot[1][i] = __fadd2_rn(tot[1][i], acc[1][i]);
    }
    float2 k1[NP], k2[NP];
    if constexpr (UNI) {
      float2 s1 = make_float2(0.f, 0.f), s2 = s1;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        s2 = __ffma2_rn(bk.ga[i], acc[0][i], s2);
        s1 = __ffma2_rn(bk.ga[i], acc[1][i], s1);
      }
      const bool leader = (lane & sl.lanes) == 0;
      const float v2 = group_lanes(s2.x + s2.y, sl.lanes);
      const float v1 = group_lanes(s1.x + s1.y, sl.lanes);
      if (leader) {
        buf[par][0][myg][warp] = v2;
        buf[par][1][myg][warp] = v1;
      }
      __syncthreads();
      float g2 = group_warps(buf[par][0], myg), g1 = group_warps(buf[par][1], myg);
      if (sl.S > 1) {
        if (slab == first) wait_started();
        if (leader && warp == 0)
          for (int k = 0; k < sl.S; ++k) {
            to_peer_f32(from + (par * sl.S + rank) * 2 * sl.kk + myg, k, g2);
            to_peer_f32(from + ((par * sl.S + rank) * 2 + 1) * sl.kk + myg, k, g1);
          }
        __syncwarp();
        cluster_arrive();
        meanwhile();
        __syncwarp();
        cluster_wait();
        g2 = g1 = 0.f;
        for (int k = 0; k < sl.S; ++k) {
          const float* fk = from + (par * sl.S + k) * 2 * sl.kk + myg;
          g2 += fk[0];
          g1 += fk[sl.kk];
        }
      } else {
        meanwhile();
      }
      const float rn = __frcp_rn(fmaxf((float)w.tb * a.cg, 1.f));
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        k1[i] = make_float2(-g1 * rn, -g1 * rn);
        k2[i] = make_float2(-g2 * rn, -g2 * rn);
      }
    } else {
      float2 both[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float2 v[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          v[i] = make_float2(0.f, 0.f);
          if (w.active) v[i] = __fmul2_rn(bk.ga[i], acc[q][i]);
        }
        if (sl.two)
          both[q] = tw.sums(v);
        else
          gather_groups<VEC>(sl, w.rows, a.cg, a.cg_div, v, scr, gs[par][q]);
      }
      if (sl.two) gather_two<VEC, 2>(sl, w.rows, a.cg, both, scr, {gs[par][0], gs[par][1]});
      if (sl.S > 1) {
        cluster_arrive();
        cluster_wait();
      }
      join_means(a, sl, w.tb, gs[par][0], gs[par][1], m1_t, m2_t);
      __syncthreads();
      if (w.active && sl.two) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          k1[i] = tw.pick(i, -m1_t[tw.g0], -m1_t[tw.g1]);
          k2[i] = tw.pick(i, -m2_t[tw.g0], -m2_t[tw.g1]);
        }
      } else if (w.active) {
        means_of<VEC>(m1_t, m2_t, c, a.cg_div, k1, k2);
      }
      meanwhile();
    }
    if (!sl.keep || !more) {  // these channels' sums leave the block
      const int row = sl.keep ? first / sl.per_sample_div : w.b;
      float* to = (float*)(part + ((long long)row * sl.S + rank) * a.C + w.c0);
      sum_channels<2, VEC>(sl, tot, scr, w.v, w.rg, w.active,
                           [&](int q, int k, float t) { to[2 * k + q] = t; });
#pragma unroll
      for (int i = 0; i < NP; ++i) tot[0][i] = tot[1][i] = make_float2(0.f, 0.f);
    }
    const auto last = bk.dx(k1, k2, w.tb == 1 && a.cg == 1);
    T* o = os + (long long)(w.t0 + w.rg) * a.xf + c;
    const T* p = x + nx.b * a.xb + nx.c0 + (long long)(nx.t0 + nx.rg) * a.xf + c;
    const T* d = dy + nx.b * a.yb + nx.c0 + (long long)(nx.t0 + nx.rg) * a.yf + c;
    auto apply = [&](int k, auto frames) {
      constexpr int U = decltype(frames)::value;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        store_ch<VEC, T>(o, last.of(load_ch<VEC, T>((const T*)(mine + (k + u) * SLOT)),
                                    load_ch<VEC, T>((const T*)(mine + half_bytes + (k + u) * SLOT))));
        o += xinc;
      }
    };
    auto fetch = [&](int k) {
      copy16(mine_a + k * SLOT, p);
      copy16(mine_a + half_bytes + k * SLOT, d);
      p += xinc;
      d += dinc;
    };
    ready = turn_over(cnt, ncnt, apply, fetch);
    w = nx;
    cnt = ncnt;
  }
  __syncwarp();
  if (sl.S > 1) {  // peers may still read this block's sums
    cluster_arrive();
    cluster_wait();
  }
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
  // (a frame's bytes and a column past its end stay within 31 bits)
  if (d->T > (1 << 20) || d->C > (1 << 28) || (long long)d->B * d->G > (1LL << 27)) return false;
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
  int grid;
  int rows;  // rows of part
  size_t smem;
};

NormCut norm_cut(const NormArgs& a, int e, int tiles, int align) {
  NormCut n{};
  // the fewest whole groups that make 64-byte pieces of a frame (16-byte
  // aligned ones) and, while there are more slabs than the SMs take twice, 16 KB:
  // a slab costs its reductions, whatever its length (250 frames of 512 channels,
  // 4096 samples: 337 us forward and 546 backward, against 433 and 780 with slabs
  // of 8 KB upward; from 32 KB upward 352 and 669).  Short of alignment, 64 channels
  // in pairs or 32.
  auto enough = [&](int k) {
    return (long long)a.T * k * a.cg * e >= 16384 || (long long)a.B * (a.G / k) <= 2 * 3 * 152;
  };
  int kk = 0;
  n.vec = 1;
  if (align == 16)
    for (int k = 1; k <= a.G && k <= MAX_KK; ++k)
      if (a.G % k == 0 && (long long)k * a.cg * e % 16 == 0) {
        // (groups as long as a thread may hold a 16-byte column of them)
        if (kk && (long long)k * a.cg * e > 16 * NT) break;
        kk = k;
        n.vec = 4;
        if (k * a.cg * e >= 64 && enough(k)) break;
      }
  if (!kk && align >= 2 * e)
    for (int k = 1; k <= a.G && k <= MAX_KK; ++k)
      if (a.G % k == 0 && k * a.cg % 2 == 0) {
        kk = k;
        n.vec = 2;
        if (k * a.cg >= 64) break;
      }
  if (!kk)
    for (int k = 1; k <= a.G && k <= MAX_KK; ++k)
      if (a.G % k == 0) {
        kk = k;
        if (k * a.cg >= 32) break;
      }
  Slab& s = n.sl;
  s.kk = kk;
  s.W = kk * a.cg;
  s.nslabs = a.B * (a.G / kk);
  const long long frame = (long long)s.W * e * tiles;
  s.S = 1;
  // resident: a thread per 16-byte column, slots within the block's share.  64 KB
  // a block keeps three blocks on an SM, and clusters go up to 16 for that: one
  // group of 512 channels, 1000 frames, 173 us forward (8 blocks of 128 KB 223,
  // from global memory 194); two groups, backward, 238 (338 from global memory).
  // (It is the slower in fp32 with one group of 384: 256 x 1000 frames, backward,
  // 381 us, 353 with 8 larger blocks.)
  const int cols16 = s.W * e / 16;
  const bool slots = n.vec == 4 && cols16 <= NT;
  auto share = [&](int S) {
    const long long per = cdiv(a.T, S);
    return slots ? cdiv(per, NT / cols16) * SLOT * tiles : per * frame;
  };
  n.res = slots && share(MAX_S) <= SHARE;
  while (s.S < (n.res ? MAX_S : 8) && share(s.S) > SHARE) s.S *= 2;
  // few slabs: shares of at least 2048 values, until there are two blocks an SM
  while (s.S < (n.res ? 8 : MAX_S) && (long long)s.nslabs * s.S < 2 * 152 &&
         (long long)a.T / (2 * s.S) * s.W >= 2048 && a.T >= 4 * s.S)
    s.S *= 2;
  s.per_max = (int)cdiv(a.T, s.S);
  if (n.res) s.slots = (int)cdiv(s.per_max, NT / cols16);
  if (n.res) n.vec = 16 / e;
  const int vr = s.W / n.vec;
  s.cbv = vr < NT ? vr : NT;
  s.pow2 = s.cbv <= 32 && (s.cbv & (s.cbv - 1)) == 0;
  for (s.lg = 0; s.lg < 5 && (kk << (s.lg + 1)) <= NT;) ++s.lg;
  s.per_sample_div = fast_div(a.G / kk);
  for (s.S_log = 0; (1 << s.S_log) < s.S;) ++s.S_log;
  for (s.step_log = 0; (2 << s.step_log) <= NT / s.cbv;) ++s.step_log;
  s.cbv_div = fast_div(s.cbv);
  n.grid = s.nslabs * s.S;
  n.rows = a.B * s.S;
  s.uni = n.res && s.pow2 && a.cg % n.vec == 0;
  s.lanes = s.uni ? 31 & ~(s.cbv - a.cg / n.vec) : 0;
  s.two = !s.uni && (a.cg >= n.vec - 1 || 2 * a.cg == n.vec);
  // shared memory: the slots, and room for the channels' and the groups' sums
  const int rows = s.pow2 ? NWARPS : NT / s.cbv;
  const size_t channels = 4 * rows * s.cbv * n.vec * tiles;
  const size_t groups = s.uni ? 0 : s.two ? 8 * NT * tiles : 4 * NT * n.vec;
  const size_t blocks = s.uni ? 16 * s.S * s.kk : 0;
  n.smem = n.res ? (size_t)s.slots * SLOT * tiles + blocks +
                       std::max(tiles > 1 ? channels : 0, groups)
                 : channels + 4 * s.cbv * n.vec * tiles;
  return n;
}

// The grid of a resident kernel: as many clusters as the card holds at a time,
// since blocks that walk slabs from the start leave nothing to later ones (512
// samples of 2000 frames: 690 us backward, against 886 where 112 clusters of 4
// were launched and 110 fit).  Where it costs at most an eighth of them, a whole
// number of samples' slabs, so that a block keeps its channels and their sums.
void norm_grid(const NormArgs& a, NormCut* n, int most) {
  Slab& s = n->sl;
  const int per_sample = a.G / s.kk;
  int clusters = std::min(s.nslabs, most);
  const int whole = clusters / per_sample * per_sample;
  s.keep = whole * 8 >= clusters * 7;
  if (s.keep) {
    clusters = whole;
    n->rows = clusters / per_sample * s.S;
  }
  n->grid = clusters * s.S;
}

// A launch in clusters of S blocks.
struct ClusterLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  ClusterLaunch(unsigned grid, int S, size_t smem, cudaStream_t st) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = S > 1 ? 1 : 0;
  }
};
template <typename... KA, typename... A>
cudaError_t launch_cluster(void (*k)(KA...), unsigned grid, int S, size_t smem, cudaStream_t st,
                           A... args) {
  const ClusterLaunch l(grid, S, smem, st);
  return cudaLaunchKernelEx(&l.cfg, k, args...);
}

// Clusters of S blocks that the card holds at a time, asked once for each kernel,
// device, cluster size and 2 KB of shared memory.
struct Resident {
  static constexpr int kStep = 2048, kSteps = (SMEM_MAX) / kStep;
  std::atomic<uint16_t> most[kDeviceSlots][5][kSteps + 1];
};
template <typename K>
cudaError_t most_clusters(K k, Resident* known, const NormCut& n, int* most) {
  const int step = (int)cdiv((long long)n.smem, Resident::kStep);
  std::atomic<uint16_t>& m = known->most[device_slot()][n.sl.S_log][step];
  *most = m.load();
  if (*most) return cudaSuccess;
  const ClusterLaunch l(n.sl.S, n.sl.S, (size_t)step * Resident::kStep, nullptr);
  cudaError_t e;
  if (n.sl.S > 1) {
    e = cudaOccupancyMaxActiveClusters(most, k, &l.cfg);
  } else {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(most, k, NT, l.cfg.dynamicSmemBytes);
    *most *= num_sms();
  }
  *most = std::min(std::max(1, *most), 65535);
  if (e == cudaSuccess) m.store((uint16_t)*most);
  return e;
}

// Shared memory above 48 KB is asked for once per kernel and device.
template <typename K>
cudaError_t opt_in(K k, std::atomic<bool>* done) {
  std::atomic<bool>& d = done[device_slot()];
  if (d.load()) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       SMEM_MAX);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) d.store(true);
  return e;
}

// dy NULL: the forward kernel, else the backward.
template <typename T, typename KF, typename KB>
cudaError_t norm_launch(KF kf, KB kb, std::atomic<bool>* fdone, std::atomic<bool>* bdone,
                        Resident* known, const NormArgs& a, NormCut* n, const void* x,
                        const void* dy, void* out, float2* part, cudaStream_t st) {
  cudaError_t e = dy ? opt_in(kb, bdone) : opt_in(kf, fdone);
  if (e != cudaSuccess) return e;
  if (known) {
    int most = 0;
    e = dy ? most_clusters(kb, known + 1, *n, &most) : most_clusters(kf, known, *n, &most);
    if (e != cudaSuccess) return e;
    norm_grid(a, n, most);
  }
  return dy ? launch_cluster(kb, n->grid, n->sl.S, n->smem, st, a, n->sl, (const T*)x,
                             (const T*)dy, (T*)out, part)
            : launch_cluster(kf, n->grid, n->sl.S, n->smem, st, a, n->sl, (const T*)x, (T*)out);
}

template <typename T, int ACT>
cudaError_t norm_launch_cut(const NormArgs& a, NormCut* n, const void* x, const void* dy,
                            void* out, float2* part, cudaStream_t st) {
  static std::atomic<bool> done[10][kDeviceSlots];
  static Resident known[4];
  if (n->res && n->sl.uni)
    return norm_launch<T>(k_norm_fwd_res<T, ACT, 1>, k_norm_bwd_res<T, ACT, 1>, done[6], done[7],
                          known, a, n, x, dy, out, part, st);
  if (n->res)
    return norm_launch<T>(k_norm_fwd_res<T, ACT, 0>, k_norm_bwd_res<T, ACT, 0>, done[0], done[1],
                          known + 2, a, n, x, dy, out, part, st);
  if (n->vec == 4)
    return norm_launch<T>(k_norm_fwd_stream<T, 4, ACT>, k_norm_bwd_stream<T, 4, ACT>, done[2],
                          done[3], nullptr, a, n, x, dy, out, part, st);
  if (n->vec == 2)
    return norm_launch<T>(k_norm_fwd_stream<T, 2, ACT>, k_norm_bwd_stream<T, 2, ACT>, done[8],
                          done[9], nullptr, a, n, x, dy, out, part, st);
  return norm_launch<T>(k_norm_fwd_stream<T, 1, ACT>, k_norm_bwd_stream<T, 1, ACT>, done[4],
                        done[5], nullptr, a, n, x, dy, out, part, st);
}

// dy NULL: forward, x -> out = y; else backward, (x, dy) -> out = dx and part.
template <typename T>
cudaError_t norm_launch_act(const NormArgs& a, NormCut* n, const void* x, const void* dy,
                            void* out, float2* part, cudaStream_t st) {
  switch (a.act) {
    case RNNT_ACT_SILU: return norm_launch_cut<T, RNNT_ACT_SILU>(a, n, x, dy, out, part, st);
    case RNNT_ACT_RELU: return norm_launch_cut<T, RNNT_ACT_RELU>(a, n, x, dy, out, part, st);
    default: return norm_launch_cut<T, RNNT_ACT_NONE>(a, n, x, dy, out, part, st);
  }
}

// Alignment of every row of x and dx, y and dy: 16 bytes, or two elements, or one.
int norm_align(const NormArgs& a, int e, const void* x, const void* y, const void* dx) {
  auto all = [&](int bytes) {
    const int v = bytes / e;
    return aligned_to(x, bytes) && aligned_to(y, bytes) && aligned_to(dx, bytes) &&
           a.xf % v == 0 && a.xb % v == 0 && a.yf % v == 0 && a.yb % v == 0;
  };
  return all(16) ? 16 : all(2 * e) ? 2 * e : e;
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
  // a row of sums for every block of a slab
  return norm_args(dims, &a) ? align_up(8 * MAX_S * (size_t)a.B * a.C + 8) : 0;
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
  NormCut n = norm_cut(a, e, 1, norm_align(a, e, x, y, nullptr));
  OPS_CHECK(e == 4 ? norm_launch_act<float>(a, &n, x, nullptr, y, nullptr, st)
                   : norm_launch_act<__nv_bfloat16>(a, &n, x, nullptr, y, nullptr, st));
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
  NormCut n = norm_cut(a, e, 2, norm_align(a, e, x, dy, dx));
  if (a.B > 0) {
    ProfScope ps("norm_bwd", st);
    OPS_CHECK(e == 4 ? norm_launch_act<float>(a, &n, x, dy, dx, part, st)
                     : norm_launch_act<__nv_bfloat16>(a, &n, x, dy, dx, part, st));
  }
  if (!dgamma && !dbeta) return RNNT_OK;
  const int rows = n.rows, S = rows > 256 ? 8 : 1;
  OPS_LAUNCH("norm_params", launch_cluster(k_norm_params, (unsigned)cdiv(a.C, 32) * S, S, 0, st,
                                           (const float2*)part, rows, a.C, S, dgamma, dbeta));
  return RNNT_OK;
}

}  // extern "C"
