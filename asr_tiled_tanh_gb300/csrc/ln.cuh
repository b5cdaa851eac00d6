// ln.cuh -- layer norm of rows: what its forward (k_ln.cu) and backward
// (k_ln_bwd.cu) kernels share (internal).
//
// A team of lanes (part of a warp, a warp or several) takes a row at a time: each lane
// holds NV units of VEC channels in registers from the load to the store, so that a row
// is read once, whatever its sums need.  Rows are copied to shared memory one to three
// ahead: a lane copies the units that it will read itself, so nothing but its own copies
// is waited for, and the loads in flight take no registers.  Blocks stay and walk the
// rows.  Both directions are bound by DRAM where a row is many units, by the steps
// between rows where it is few: 1024 x 1000 rows of 512 in bf16, ragged, 274 us forward
// and 380 backward (0.93 and 0.94 of a plain copy's rate), 512 x 2000 rows of 24 28 and
// 53 (0.51 and 0.41).
#pragma once
#include <algorithm>
#include <atomic>

#include "ops.h"
#include "ptx.cuh"

namespace rnnt {
namespace ln {

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

// Row r of the batch (where it is taken by a block).
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

// 1 / sqrt(var): rsqrtf is 2 ulp off, the step leaves it within one.  NaN for 0 and for
// infinity (a row of one value without eps, squares past the range), by 0 * inf in the step.
__device__ __forceinline__ float root_of(float var) {
  const float r = rsqrtf(var);
  return fmaf(0.5f * r, fmaf(-var * r, r, 1.f), r);
}

// Whether a row's deviation may be the rounding of its mean: squares about it that come to
// 2^-22 of its own or less.  A sum of equal terms is rounded where their multiples need more
// bits than fp32 has, by up to 2^-14 of itself in the widest rows, and a row of one value had
// deviations of that size.  The mean of what is left about the first (those differences are
// exact) corrects it, and the squares are added again; other rows keep their bits.  (The
// branch costs 0 to 1% of the forward where rows are many, 0.4 us of 7.4 for 16 x 400 x
// 1024, fp32 to bf16; teams' bf16 rows, where it would be 5 to 12%, do not need it.)
__device__ __forceinline__ bool may_be_flat(float squares, float rC, float mean) {
  const float m = mean * 0x1p-11f;
  return squares > 0.f && squares * rC < m * m;
}

// ---- vectors ------------------------------------------------------------------
// VEC (8, 4 or 2) channels next to each other, or two that are as many channels apart
// as the team has lanes (VEC = 1: rows of odd width or place), as pairs of fp32.
constexpr int kPairs(int vec) { return vec == 1 ? 1 : vec / 2; }
template <int VEC>
struct Vals {
  float2 p[kPairs(VEC)];
  __device__ __forceinline__ void fill(float v) {
#pragma unroll
    for (int i = 0; i < kPairs(VEC); ++i) p[i] = make_float2(v, v);
  }
};

template <typename W> struct Two { W a, b; };
template <int VEC, int SIZE> struct UnitOf;
template <> struct UnitOf<1, 2> { using type = Two<unsigned short>; };
template <> struct UnitOf<1, 4> { using type = Two<uint32_t>; };
template <> struct UnitOf<2, 2> { using type = uint32_t; };
template <> struct UnitOf<2, 4> { using type = uint2; };
template <> struct UnitOf<4, 2> { using type = uint2; };
template <> struct UnitOf<4, 4> { using type = uint4; };
template <> struct UnitOf<8, 2> { using type = uint4; };
// as they are stored
template <int VEC, typename T>
using Unit = typename UnitOf<VEC, (int)sizeof(T)>::type;

template <int VEC, typename T>
__device__ __forceinline__ Vals<VEC> widen(const Unit<VEC, T>& u) {
  Vals<VEC> v;
  if constexpr (VEC == 1 && sizeof(T) == 2) {
    v.p[0] = make_float2(__uint_as_float((uint32_t)u.a << 16),
                         __uint_as_float((uint32_t)u.b << 16));
  } else if constexpr (VEC == 1) {
    v.p[0] = make_float2(__uint_as_float(u.a), __uint_as_float(u.b));
  } else if constexpr (sizeof(T) == 4) {
    const float* f = (const float*)&u;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) v.p[i] = make_float2(f[2 * i], f[2 * i + 1]);
  } else {
    const uint32_t* w = (const uint32_t*)&u;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) v.p[i] = make_float2(ptx::bf16lo(w[i]), ptx::bf16hi(w[i]));
  }
  return v;
}

// A lane's units of a row: unit j begins at channel at(j).
template <int VEC>
struct Cols {
  int lane, lanes, C;
  __device__ __forceinline__ int at(int j) const {
    return VEC == 1 ? lane + 2 * j * lanes : (lane + j * lanes) * VEC;
  }
  __device__ __forceinline__ bool has(int j) const { return at(j) < C; }
  // (the second of two that are apart)
  __device__ __forceinline__ bool both(int j) const {
    return VEC == 1 ? at(j) + lanes < C : has(j);
  }
  template <typename T>
  __device__ __forceinline__ Vals<VEC> load(const T* row, int j) const {
    const T* from = row + at(j);
    if constexpr (VEC == 1) {
      Vals<1> v;
      v.p[0] = make_float2(to_f<T>(from[0]), both(j) ? to_f<T>(from[lanes]) : 0.f);
      return v;
    } else {
      return widen<VEC, T>(*(const Unit<VEC, T>*)from);
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int j, const Vals<VEC>& v) const {
    if (!has(j)) return;
    T* to = row + at(j);
    if constexpr (VEC == 1) {
      to[0] = from_f<T>(v.p[0].x);
      if (both(j)) to[lanes] = from_f<T>(v.p[0].y);
    } else {
      Unit<VEC, T> u;
      if constexpr (sizeof(T) == 4) {
        float* f = (float*)&u;
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          f[2 * i] = v.p[i].x;
          f[2 * i + 1] = v.p[i].y;
        }
      } else {
        uint32_t* w = (uint32_t*)&u;
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) w[i] = ptx::pack_bf16x2(v.p[i].x, v.p[i].y);
      }
      *(Unit<VEC, T>*)to = u;
    }
  }
  // fp32 parameters of unit j (NULL: all `other`; 0 past the row's end)
  __device__ __forceinline__ Vals<VEC> param(const float* p, int j, float other, bool al16) const {
    Vals<VEC> v;
    v.fill(0.f);
    if (!has(j)) return v;
    if (!p) {
      v.fill(other);
    } else if constexpr (VEC == 1) {
      v.p[0] = make_float2(__ldg(p + at(j)), both(j) ? __ldg(p + at(j) + lanes) : 0.f);
    } else if (VEC >= 4 && al16) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const float4 q = __ldg((const float4*)(p + at(j)) + i);
        v.p[2 * i] = make_float2(q.x, q.y);
        v.p[2 * i + 1] = make_float2(q.z, q.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPairs(VEC); ++i)
        v.p[i] = make_float2(__ldg(p + at(j) + 2 * i), __ldg(p + at(j) + 2 * i + 1));
    }
    return v;
  }
};

// ---- a block a row ------------------------------------------------------------
// Rows too wide for a team: read again for each of their sums (from L2).
constexpr int WT = 512, WWARPS = WT / 32;

// Sums of two values over the block, for all threads.
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

// ---- teams ----------------------------------------------------------------------
constexpr int MAX_THREADS = 512;
constexpr int STAGES = 3;  // at most

// A row is taken by part of a warp (4, 8 or 16 lanes), a warp, or several.
enum { PART = 0, WARP = 1, WARPS = 2 };

struct Team {
  int lanes;    // threads a row
  int teams;    // a block's
  FastDiv div;  // by lanes
};

// The calling thread's place.
struct Place {
  int team, lane;   // in the block, in the team
  int first, step;  // rows first, first + step, ... are the team's
};
template <int MODE>
__device__ __forceinline__ Place place_of(const Team& t) {
  Place p;
  p.team = MODE == WARP ? threadIdx.x >> 5 : (int)threadIdx.x / t.div;
  p.lane = MODE == WARP ? threadIdx.x & 31 : threadIdx.x - p.team * t.lanes;
  p.first = blockIdx.x * t.teams + p.team;
  p.step = gridDim.x * t.teams;
  return p;
}

// Sums of NQ values over the team, for all its lanes, in a fixed order.  scr: one
// of two buffers in turn, so that one barrier a sum keeps writers off readers.
template <int MODE, int NQ>
__device__ __forceinline__ void team_sum(float (&v)[NQ], const Team& t, const Place& p,
                                         float (*scr)[NQ]) {
#pragma unroll
  for (int d = 16; d; d >>= 1)
    if (MODE != PART || d < t.lanes)
#pragma unroll
      for (int q = 0; q < NQ; ++q) v[q] += __shfl_xor_sync(0xffffffffu, v[q], d);
  if constexpr (MODE == WARPS) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = t.lanes >> 5;
    if (lane == 0)
#pragma unroll
      for (int q = 0; q < NQ; ++q) scr[warp][q] = v[q];
    ptx::named_barrier(1 + p.team, t.lanes);
#pragma unroll
    for (int q = 0; q < NQ; ++q) v[q] = lane < warps ? scr[p.team * warps + lane][q] : 0.f;
#pragma unroll
    for (int d = 8; d; d >>= 1)
      if (d < warps)
#pragma unroll
        for (int q = 0; q < NQ; ++q) v[q] += __shfl_xor_sync(0xffffffffu, v[q], d);
#pragma unroll
    for (int q = 0; q < NQ; ++q) v[q] = __shfl_sync(0xffffffffu, v[q], 0);
  }
}

// ---- a team's rows, one after another --------------------------------------------
// Steps of the walk, by additions alone.
struct Stride {
  int db, dt;
  __device__ __forceinline__ Stride(const LnArgs& a, int step) {
    db = step / a.t_div;
    dt = step - db * a.T;
  }
};
struct Walk {
  int b, t;
  __device__ __forceinline__ Walk(const LnArgs& a, int r) {
    b = r / a.t_div;
    t = r - b * a.T;
  }
};
// An offset that goes with a walk: by `step` a row, and by `wrap` where a sample ends.
struct Offset {
  long long at, step, wrap;
  __device__ __forceinline__ Offset(const LnArgs& a, const Walk& w, const Stride& s, long long f,
                                    long long b) {
    at = w.b * b + w.t * f;
    step = s.db * b + s.dt * f;
    wrap = b - a.T * f;
  }
};
template <typename... O>
__device__ __forceinline__ void advance(const LnArgs& a, const Stride& s, Walk& w, O&... o) {
  w.b += s.db;
  w.t += s.dt;
  ((o.at += o.step), ...);
  if (w.t >= a.T) {
    w.t -= a.T;
    ++w.b;
    ((o.at += o.wrap), ...);
  }
}
// Length of the walk's sample, asked for ahead of its use.
__device__ __forceinline__ int ask_length(const LnArgs& a, const Walk& w) {
  return a.lengths && w.b < a.B ? __ldg(a.lengths + w.b) : a.T - a.extra;
}
// Whether the walk's row exists by that length.
__device__ __forceinline__ bool exists(const LnArgs& a, const Walk& w, int length, bool says) {
  if (w.b >= a.B) return false;
  if ((unsigned)length > (unsigned)(a.T - a.extra)) {
    if (says) report(a.status, RNNT_ERR_LENGTH_RANGE);
    return false;
  }
  return w.t < length + a.extra;
}

// ---- rows ahead -------------------------------------------------------------------
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A lane's units of one tensor's rows ahead: [S stages][NV][threads], those past the
// row's end zero.  A stage is read and then filled again.  Elements of two bytes are
// too small for the copies: units of two such are loaded to registers instead, one
// row ahead.
template <int VEC, typename T>
constexpr bool kCopied = VEC * sizeof(T) >= 4;
template <int VEC, int NV, int S, typename T>
struct Ring {
  using U = Unit<VEC, T>;
  static constexpr int BYTES = sizeof(U);
  unsigned char* mine;
  int pitch;  // bytes from one of a lane's units to its next
  U held[kCopied<VEC, T> ? 1 : NV];
  static __host__ __device__ size_t bytes(int threads) {
    return kCopied<VEC, T> ? (size_t)S * NV * threads * BYTES : 0;
  }
  // (a barrier between this and the first copies)
  __device__ __forceinline__ void init(unsigned char* smem) {
    if constexpr (kCopied<VEC, T>) {
      mine = smem + threadIdx.x * BYTES;
      pitch = blockDim.x * BYTES;
#pragma unroll
      for (int k = 0; k < S * NV; ++k) *(U*)(mine + k * pitch) = U{};
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) held[j] = U{};
    }
  }
  __device__ __forceinline__ void fetch(int stage, const T* row, const Cols<VEC>& c) {
    const uint32_t to = kCopied<VEC, T> ? ptx::smem_u32(mine) + stage * (NV * pitch) : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const T* from = row + c.at(j);
      if constexpr (!kCopied<VEC, T>) {
        if (c.has(j)) held[j].a = *(const unsigned short*)from;
        if (c.both(j)) held[j].b = *(const unsigned short*)(from + c.lanes);
      } else if constexpr (VEC == 1) {
        if (c.has(j)) copy_async<4>(to + j * pitch, from);
        if (c.both(j)) copy_async<4>(to + j * pitch + 4, from + c.lanes);
      } else {
        if (c.has(j)) copy_async<BYTES>(to + j * pitch, from);
      }
    }
  }
  __device__ __forceinline__ void read(U (&u)[NV], int stage) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (kCopied<VEC, T>) u[j] = *(const U*)(mine + (stage * NV + j) * pitch);
      else u[j] = held[j];
    }
  }
};

// ---- host -------------------------------------------------------------------------
// Lanes for rows of n units, and nv units a lane among the numbers that are compiled: at
// most `one` of a warp that holds a row, `two` of two, `most` of more; 0 lanes: too wide.  Of units
// of 16 bytes those that cost least: a lane's steps for a row count as 2.2 times those
// for a unit, and what a block of 256 threads has left over is lost.  So a warp's steps
// between rows serve several where it can hold them, and few lanes idle (bf16, us: 512 x
// 2000 rows of 256 in 16 lanes of two units 159 forward and 253 backward, in 32 of one
// 181 and 324; 256 x 1000 rows of 1280 in two warps of 3 units 216 forward, in three of 2
// 313; 2000 in four of 2 367, in three of 3 395).
constexpr int PART_UNITS = 3;  // of part of a warp
inline Team team_for(int n, int one, int two, int most, bool wide_units, int* nv) {
  Team t{};
  if (wide_units) {
    long long least = 0;
    auto offer = [&](long long lanes, long long threads, int per) {
      const long long cost = threads * (11 + 5 * per);
      if (lanes * per < n || (least && cost >= least)) return;
      least = cost;
      t.lanes = (int)lanes;
      *nv = per;
    };
    for (int lanes = 4; lanes <= 16; lanes *= 2)
      for (int per = 1; per <= std::min(one, PART_UNITS); ++per) offer(lanes, lanes, per);
    for (int per = 2; per <= one; ++per) offer(32, 32, per);
    for (int per = 2; per <= most; ++per) {
      const long long w = std::max(2LL, cdiv(n, 32LL * per));
      if (32 * w <= MAX_THREADS) offer(32 * w, w > 8 ? 32 * w : 256 / (8 / w), per);
    }
    for (int per = most + 1; per <= two; ++per) offer(64, 64, per);
  } else {
    const long long w = cdiv(n, 32LL * most);
    if (32 * w <= MAX_THREADS) t.lanes = (int)(32 * w);
    if (w == 1)
      while (t.lanes > 4 && n <= t.lanes / 2 * 2) t.lanes /= 2;
    if (t.lanes) *nv = ((int)cdiv(n, t.lanes) + 1) / 2 * 2;
  }
  if (!t.lanes) return t;
  t.teams = t.lanes > 256 ? 1 : 256 / t.lanes;
  t.div = fast_div(t.lanes);
  return t;
}

// f.run<VEC, NV, MODE>(team) for rows of C channels in units of vec (V16: those of 16
// bytes): at most CH channels a lane, CH1 of a warp that holds a row, CH2 of two, ONE
// pairs of those apart; false: no team holds such a row.
template <int VEC, int NV, typename F>
cudaError_t by_mode(const Team& t, const F& f) {
  constexpr bool PARTS = NV <= (VEC >= 4 ? PART_UNITS : 2);
  if (PARTS && t.lanes < 32) return f.template run<VEC, NV, PARTS ? PART : WARP>(t);
  if (t.lanes == 32) return f.template run<VEC, NV, WARP>(t);
  return f.template run<VEC, NV, WARPS>(t);
}
template <int VEC, int NV, int MOST1, int MOST2, int MOST, typename F>
cudaError_t by_units(const Team& t, int nv, const F& f) {
  if constexpr (NV == 1) {
    if (nv == 1) return f.template run<VEC, 1, PART>(t);
  } else if constexpr (NV <= MOST) {
    if (nv == NV) return by_mode<VEC, NV>(t, f);
  } else if (nv == NV) {
    if (NV <= PART_UNITS && t.lanes < 32)
      return f.template run<VEC, NV, NV <= PART_UNITS ? PART : WARP>(t);
    if (NV <= MOST2 && t.lanes > 32) return f.template run<VEC, NV, NV <= MOST2 ? WARPS : WARP>(t);
    return f.template run<VEC, NV, WARP>(t);
  }
  if constexpr (NV < MOST1) return by_units<VEC, NV + 1, MOST1, MOST2, MOST>(t, nv, f);
  return cudaErrorInvalidValue;
}
template <int VEC, int MOST, typename F>
cudaError_t by_pairs(const Team& t, int nv, const F& f) {
  if (nv == 2) return by_mode<VEC, 2>(t, f);
  if (nv == 4) return by_mode<VEC, 4>(t, f);
  if (MOST == 6 || nv == 6) return by_mode<VEC, 6>(t, f);
  return by_mode<VEC, MOST>(t, f);
}
template <int V16, int CH1, int CH2, int CH, int ONE, typename F>
bool by_team(int C, int vec, const F& f, cudaError_t* e) {
  constexpr int MOST1 = CH1 / V16, MOST2 = CH2 / V16, MOST = CH / V16;
  const bool wide = vec == V16;
  int nv = 0;
  const int narrow = vec == 2 ? 8 : ONE;
  const Team t = team_for((int)cdiv(C, vec == 1 ? 2 : vec), wide ? MOST1 : narrow,
                          wide ? MOST2 : narrow, wide ? MOST : narrow, wide, &nv);
  if (!t.lanes) return false;
  if (wide) *e = by_units<V16, 1, MOST1, MOST2, MOST>(t, nv, f);
  else *e = vec == 2 ? by_pairs<2, 8>(t, nv, f) : by_pairs<1, ONE>(t, nv, f);
  return true;
}

// Vector width that every row of these tensors allows: 16 bytes of the larger
// type, two elements, or one.
inline int vec_of(const LnArgs& a, int ex, const void* x, const void* dx, int ey, const void* y) {
  auto all = [&](int v) {
    return a.C % v == 0 && a.xf % v == 0 && a.yf % v == 0 &&
           (a.B <= 1 || (a.xb % v == 0 && a.yb % v == 0)) && aligned_to(x, v * ex) &&
           aligned_to(dx, v * ex) && aligned_to(y, v * ey);
  };
  const int v16 = 16 / std::max(ex, ey);
  return all(v16) ? v16 : all(2) ? 2 : 1;
}

// Most of a kernel's blocks that an SM holds: asked once per kernel, device and
// number of warps (a kernel's shared memory follows from its threads).
struct Known {
  std::atomic<uint8_t> blocks[kDeviceSlots][MAX_THREADS / 32 + 1];
};
constexpr int SMEM_MAX = 200 * 1024;
template <typename K>
cudaError_t blocks_per_sm(K k, Known* known, int threads, size_t smem, int* out) {
  std::atomic<uint8_t>& m = known->blocks[device_slot()][threads / 32];
  *out = m.load();
  if (*out) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, k, threads, smem);
  if (e != cudaSuccess) return e;
  *out = std::max(1, *out);
  m.store((uint8_t)*out);
  return e;
}

// launchers (k_ln.cu, k_ln_bwd.cu); part_rows: rows of part that were written
int part_rows_max(const LnArgs& a);
cudaError_t launch_bwd(const LnArgs& a, int x_dtype, int y_dtype, const void* x, const void* dy,
                       void* dx, float2* part, int* part_rows, bool params, cudaStream_t st);
cudaError_t launch_params(const float2* part, int rows, int C, float* dgamma, float* dbeta,
                          cudaStream_t st);

}  // namespace ln
}  // namespace rnnt
