// k_orth.cu -- orthogonalised update by Newton-Schulz products
// (include/rnnt_ops.h).
//
// With X the scaled matrix, m its shorter and n its longer side, a step is
//   gram    S = X X^T        (m x m, over n; X^T X when the rows are longer)
//   poly    P = b S + c S S - d I
//   update  X <- (a + d) X + P X
// One kernel runs all steps: it is persistent (one block per SM at most, all of
// them resident: a cooperative launch), its blocks take 128-wide tiles of each
// product in turn, and a grid barrier separates the products, which depend on
// one another throughout.  Separate launches would pay 15 times for tensor
// memory, barriers and pipeline fill.
//
// Numbers.  The tensor cores multiply fp16 (11 bits) and add in fp32.  X, S and
// P are kept as two fp16 values each, hi = fp16(v 2^k) and lo = fp16(v 2^k - hi):
// 22 bits, with a fixed k, since the iterate's entries stay below 1.3, those of
// S below 1.5 and those of P below 4 (a singular value never leaves [0, 1.21]).
// A product takes one term (hi hi) or three (hi hi + hi lo + lo hi, the missing
// lo lo is below 2^-22):
//   exact (fp32 results, and small matrices, where it costs nothing): three
//     terms everywhere;
//   fast (bf16 results): one term in gram and update, whose rounding of 2^-12
//     per entry averages out over the row; three in poly, the smallest product,
//     because b S and c S S largely cancel near a singular value of 1.  For the
//     same reason P is taken off its mean there: for singular values near 1 its
//     diagonal is about d = b + c ... = -2.5, which the update applies in fp32
//     through (a + d) X.  The shift enters as the steps converge (it would cost
//     small singular values digits in the first ones).  In 64-bit emulation over
//     flat, 1/i^p and low-rank-plus-noise spectra the fast result is 0.3 to
//     1.6e-3 off, next to 1.7e-3 for its own rounding to bf16.
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "ops.h"
#include "ptx.cuh"

namespace rnnt {
namespace {

// The Muon optimiser's quintic.
constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;

constexpr int BM = 128, BK = 64;      // tile rows; K per stage: a 128-byte swizzle atom of fp16
constexpr int BN_MAX = 256;
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK * 2, STAGE_BYTES = A_BYTES + BN_MAX * BK * 2;
constexpr int EPI_WARPS = 8, THREADS = 64 + 32 * EPI_WARPS;
constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + 256;
constexpr uint64_t WAIT_NS = 2000000000ull;  // 2 s per wait, then give up
constexpr int XE = 14, SE = 14, PE = 13;     // scale exponents of X, S and P

enum { GRAM, POLY, UPDATE };

struct OrthMaps {  // X buffers 0 and 1, S, P; hi and lo of each
  CUtensorMap m[4][2];
};
enum { BUF_X0, BUF_X1, BUF_S, BUF_P };

struct OrthArgs {
  int m, n, tall, batch, steps;
  int terms;            // of gram and update: 3 (exact) or 1 (fast)
  int rows, cols;       // of G, and of X
  long long ldx, ldm;   // row strides of X; of S and P
  __half* X[2][2];
  __half* S[2];
  __half* P[2];
  float* part;          // gram partial tiles [splits][batch][tiles][128][128]
  int tiles;            // 128 x 128 tiles on and above the diagonal of S
  int splits, kb_split; // gram: K ranges and their length in K blocks
  int bn;               // update: tile width
  int ut_m, ut_n;       // update: tiles
  const void* G;
  int in_f32;
  long long in_ld, in_batch;
  void* O;
  int out_f32;
  long long out_ld, out_batch;
  float eps;
  const double* sums;   // [batch][nb] partial sums of squares
  int nb;
  unsigned* counter;    // grid barrier: arrivals so far
  int* abort;
  int32_t* status;
};

// ---- sums of squares ---------------------------------------------------------------
// Block (i, b) adds the squares of its share of matrix b: eight at a time in
// fp32, those in fp64, so that neither 1e-18 nor 1e18 leaves the range.  Also
// clears the barrier of the kernel that follows.
template <typename T>
__global__ void __launch_bounds__(256)
k_orth_sumsq(OrthArgs a, double* sums) {
  __shared__ double part[8];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    *a.counter = 0;
    *a.abort = 0;
  }
  const T* g = (const T*)a.G + blockIdx.y * a.in_batch;
  const int chunks = (a.cols + 7) / 8;  // of eight columns
  const bool vec = a.cols % 8 == 0 && a.in_ld % 8 == 0 && a.in_batch % 8 == 0 &&
                   ((uintptr_t)a.G & 15) == 0;
  double s = 0;
  const long long total = (long long)a.rows * chunks;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const int r = (int)(i / chunks), c = (int)(i - (long long)r * chunks) * 8;
    const T* p = g + r * a.in_ld + c;
    float q = 0.f;
    if (vec) {
      if constexpr (sizeof(T) == 4) {
        const float4 x = __ldg((const float4*)p), y = __ldg((const float4*)p + 1);
        q = x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w + y.x * y.x + y.y * y.y + y.z * y.z +
            y.w * y.w;
      } else {
        const uint4 x = __ldg((const uint4*)p);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float lo = ptx::bf16lo(w[k]), hi = ptx::bf16hi(w[k]);
          q += lo * lo + hi * hi;
        }
      }
    } else {
      for (int k = 0; k < 8 && c + k < a.cols; ++k) {
        const float v = to_f<T>(p[k]);
        q += v * v;
      }
    }
    s += (double)q;
  }
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0;
    for (int k = 0; k < 8; ++k) s += part[k];
    sums[blockIdx.y * (long long)gridDim.x + blockIdx.x] = s;
  }
}

// ---- pieces --------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(m), "r"(ptx::smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// global writes of this thread become visible to TMA loads ordered after them
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *(const uint32_t*)&h;
}
__device__ __forceinline__ float2 unpack_h2(uint32_t w) { return __half22float2(*(__half2*)&w); }

// hi and lo of two scaled values
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_h2(x, y);
  const float2 f = unpack_h2(hi);
  lo = pack_h2(x - f.x, y - f.y);
}

// Instruction descriptor of tcgen05.mma kind::f16 with fp16 operands, fp32
// accumulation, M = 128.
__device__ __forceinline__ uint32_t idesc_f16(int bn, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

// Diagonal shift of P in step k (see the head of this file).
__device__ __forceinline__ float shift_of(int k) {
  return k < 2 ? 0.f : k == 2 ? -0.7f : k == 3 ? -2.2f : -2.5f;
}

// Tile t of the upper triangle of an nt x nt grid of tiles, row by row.
__device__ __forceinline__ void triangle(int t, int nt, int& i, int& j) {
  i = 0;
  while (t >= nt - i) {
    t -= nt - i;
    ++i;
  }
  j = i + t;
}

// One product: its tiles and operands.
struct Work {
  int kind, units, kbs, K, bn, terms, a_mn, b_mn, a_buf, b_buf;
};
struct Unit {
  int b, m0, n0, kb0, kb1, tile, diag;
};

__device__ __forceinline__ Work work_of(const OrthArgs& a, int kind, int cur) {
  Work w;
  w.kind = kind;
  w.a_mn = w.b_mn = 0;
  w.bn = 128;
  w.terms = a.terms;
  if (kind == GRAM) {
    w.K = a.n;
    w.a_buf = w.b_buf = cur;
    w.a_mn = w.b_mn = a.tall;
    w.units = a.batch * a.tiles * a.splits;
  } else if (kind == POLY) {
    w.K = a.m;
    w.a_buf = w.b_buf = BUF_S;
    w.terms = 3;
    w.units = a.batch * a.tiles;
  } else {
    w.K = a.m;
    w.bn = a.bn;
    w.a_buf = a.tall ? cur : BUF_P;
    w.b_buf = a.tall ? BUF_P : cur;
    w.b_mn = !a.tall;
    w.units = a.batch * a.ut_m * a.ut_n;
  }
  w.kbs = (w.K + BK - 1) / BK;
  return w;
}

__device__ __forceinline__ Unit unit_of(const OrthArgs& a, const Work& w, int u) {
  Unit q;
  q.kb0 = 0;
  q.kb1 = w.kbs;
  q.tile = u;
  q.diag = 0;
  if (w.kind == UPDATE) {
    const int n = u % a.ut_n, rest = u / a.ut_n;
    q.b = rest / a.ut_m;
    q.m0 = (rest - q.b * a.ut_m) * BM;
    q.n0 = n * w.bn;
    return q;
  }
  int rest = u;
  if (w.kind == GRAM) {
    const int per = a.batch * a.tiles, ks = u / per;
    rest = u - ks * per;
    q.kb0 = ks * a.kb_split;
    q.kb1 = min(w.kbs, q.kb0 + a.kb_split);
  }
  q.b = rest / a.tiles;
  int i, j;
  triangle(rest - q.b * a.tiles, (a.m + BM - 1) / BM, i, j);
  q.m0 = i * BM;
  q.n0 = j * BM;
  q.diag = i == j;
  return q;
}

// Wait until `target` blocks have arrived at the grid barrier in all.
__device__ __forceinline__ bool grid_wait(const OrthArgs& a, unsigned target,
                                          volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (int i = 0;; ++i) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a.counter) : "memory");
    if (v >= target) return true;
    if ((i & 63) == 63) {
      if (*abort_flag || *(volatile int*)a.abort) return false;
      const uint64_t t = ptx::globaltimer();
      if (!t0) t0 = t;
      if (t - t0 > WAIT_NS) return false;
    }
  }
}

__device__ __forceinline__ void give_up(const OrthArgs& a, volatile int* abort_flag) {
  *abort_flag = 1;
  atomicExch(a.abort, 1);
  report(a.status, RNNT_ERR_TIMEOUT);
}

// Barrier of the epilogue warps; whether any of their threads said so.
__device__ __forceinline__ bool epi_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred P, Q;\n setp.ne.u32 P, %1, 0;\n"
      " barrier.cta.red.or.pred Q, 1, %2, P;\n selp.u32 %0, 1, 0, Q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(32 * EPI_WARPS)
      : "memory");
  return r != 0;
}

// 32 consecutive values of a row as hi and lo planes; nv of them exist.
__device__ __forceinline__ void store_split(__half* hi, __half* lo, const float (&v)[32], int nv) {
  if (nv >= 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 h, l;
      split2(v[8 * i], v[8 * i + 1], h.x, l.x);
      split2(v[8 * i + 2], v[8 * i + 3], h.y, l.y);
      split2(v[8 * i + 4], v[8 * i + 5], h.z, l.z);
      split2(v[8 * i + 6], v[8 * i + 7], h.w, l.w);
      *(uint4*)(hi + 8 * i) = h;
      *(uint4*)(lo + 8 * i) = l;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    uint32_t h, l;
    split2(v[2 * i], v[2 * i + 1], h, l);
    if (2 * i < nv) {
      ((unsigned short*)hi)[2 * i] = (unsigned short)h;
      ((unsigned short*)lo)[2 * i] = (unsigned short)l;
    }
    if (2 * i + 1 < nv) {
      ((unsigned short*)hi)[2 * i + 1] = (unsigned short)(h >> 16);
      ((unsigned short*)lo)[2 * i + 1] = (unsigned short)(l >> 16);
    }
  }
}

// The transposed copy: value j goes to row j of the planes, at this lane's
// column (a warp's lanes are 32 neighbouring columns).
__device__ __forceinline__ void store_split_t(__half* hi, __half* lo, long long ld,
                                              const float (&v)[32], int nv) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    uint32_t h, l;
    split2(v[2 * i], v[2 * i + 1], h, l);
    if (2 * i < nv) {
      ((unsigned short*)hi)[2 * i * ld] = (unsigned short)h;
      ((unsigned short*)lo)[2 * i * ld] = (unsigned short)l;
    }
    if (2 * i + 1 < nv) {
      ((unsigned short*)hi)[(2 * i + 1) * ld] = (unsigned short)(h >> 16);
      ((unsigned short*)lo)[(2 * i + 1) * ld] = (unsigned short)(l >> 16);
    }
  }
}

// v[j] = hi + lo (scaled) of 32 consecutive values; 0 past nv.
__device__ __forceinline__ void load_split(const __half* hi, const __half* lo, float (&v)[32],
                                           int nv) {
  if (nv >= 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 h = *(const uint4*)(hi + 8 * i), l = *(const uint4*)(lo + 8 * i);
      const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = unpack_h2(hw[k]), y = unpack_h2(lw[k]);
        v[8 * i + 2 * k] = x.x + y.x;
        v[8 * i + 2 * k + 1] = x.y + y.y;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 32; ++j)
    v[j] = j < nv ? __half2float(hi[j]) + __half2float(lo[j]) : 0.f;
}

// One 32-column piece of an accumulator row: v holds the products of row
// `row`, columns col0 .. col0 + 31.
__device__ __forceinline__ void finish(const OrthArgs& a, const Work& w, const Unit& q, int step,
                                       int cur, float (&v)[32], int row, int col0, int lrow,
                                       int lcol) {
  if (w.kind == UPDATE) {
    const int nv = min(32, a.cols - col0);
    if (row >= a.rows || nv <= 0) return;
    const long long at = ((long long)q.b * a.rows + row) * a.ldx + col0;
    float x[32];
    load_split(a.X[cur][0] + at, a.X[cur][1] + at, x, nv);
    const float f = kA + shift_of(step);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = fmaf(f, x[j], v[j] * (1.f / (1 << PE)));
    if (step + 1 < a.steps) {
      store_split(a.X[cur ^ 1][0] + at, a.X[cur ^ 1][1] + at, v, nv);
      return;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= 1.f / (1 << XE);
    const long long o = q.b * a.out_batch + row * a.out_ld + col0;
    if (a.out_f32) {
      float* p = (float*)a.O + o;
      if (nv == 32 && ((uintptr_t)p & 15) == 0) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *(float4*)(p + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < nv) p[j] = v[j];
      }
    } else {
      __nv_bfloat16* p = (__nv_bfloat16*)a.O + o;
      if (nv == 32 && ((uintptr_t)p & 15) == 0) {
#pragma unroll
        for (int j = 0; j < 32; j += 8)
          *(uint4*)(p + j) = make_uint4(
              ptx::pack_bf16x2(v[j], v[j + 1]), ptx::pack_bf16x2(v[j + 2], v[j + 3]),
              ptx::pack_bf16x2(v[j + 4], v[j + 5]), ptx::pack_bf16x2(v[j + 6], v[j + 7]));
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < nv) p[j] = __float2bfloat16_rn(v[j]);
      }
    }
    return;
  }
  if (w.kind == GRAM && a.splits > 1) {
    float* p = a.part + (long long)q.tile * (BM * BM) + lrow * BM + lcol;
#pragma unroll
    for (int j = 0; j < 32; j += 4)
      *(float4*)(p + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    return;
  }
  const int nv = min(32, a.m - col0);
  if (row >= a.m || nv <= 0) return;
  const long long base = (long long)q.b * a.m * a.ldm, at = base + row * a.ldm + col0;
  __half *hi = a.S[0], *lo = a.S[1];
  if (w.kind == GRAM) {
    const float f = 1.f / (1 << (2 * XE - SE));
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= f;
  } else {
    float s[32];
    load_split(a.S[0] + at, a.S[1] + at, s, nv);
    const float fs = kB / (1 << (SE - PE)), fp = kC / (1 << (2 * SE - PE));
    const float d = shift_of(step) * (1 << PE);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      v[j] = fmaf(fs, s[j], v[j] * fp) - (row == col0 + j ? d : 0.f);
    hi = a.P[0];
    lo = a.P[1];
  }
  store_split(hi + at, lo + at, v, nv);
  if (!q.diag) {
    const long long t = base + col0 * a.ldm + row;
    store_split_t(hi + t, lo + t, a.ldm, v, nv);
  }
}

// 1 / (|G|_F + eps) of matrix b, the same in every lane (0 for a matrix of
// zeros with eps = 0, NaN when the norm is not finite).
__device__ __forceinline__ float inverse_norm(const OrthArgs& a, int b) {
  const int lane = threadIdx.x & 31;
  double s = 0;
  for (int i = lane; i < a.nb; i += 32) s += a.sums[(long long)b * a.nb + i];
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (!isfinite(s)) return __int_as_float(0x7fc00000);
  const float n = (float)sqrt(s) + a.eps;
  return n > 0.f ? 1.f / n : 0.f;
}

// X = G / (|G|_F + eps) as hi and lo planes (epilogue warps of all blocks).
template <typename T>
__device__ __forceinline__ void convert(const OrthArgs& a, int tid, int nthreads) {
  const int chunks = (a.cols + 7) / 8;
  const bool vec = a.cols % 8 == 0 && a.in_ld % 8 == 0 && a.in_batch % 8 == 0 &&
                   ((uintptr_t)a.G & 15) == 0;
  const long long per = (long long)a.rows * chunks;
  for (int b = 0; b < a.batch; ++b) {
    const float f = inverse_norm(a, b) * (1 << XE);
    for (long long i = tid; i < per; i += nthreads) {
      const int r = (int)(i / chunks), c = (int)(i - (long long)r * chunks) * 8;
      const T* p = (const T*)a.G + b * a.in_batch + r * a.in_ld + c;
      const int nv = min(8, a.cols - c);
      float v[8];
      if (vec) {
        if constexpr (sizeof(T) == 4) {
          const float4 x = __ldg((const float4*)p), y = __ldg((const float4*)p + 1);
          v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
          v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
        } else {
          const uint4 x = __ldg((const uint4*)p);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[2 * k] = ptx::bf16lo(w[k]);
            v[2 * k + 1] = ptx::bf16hi(w[k]);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < nv ? to_f<T>(p[k]) : 0.f;
      }
      uint4 h, l;
      split2(v[0] * f, v[1] * f, h.x, l.x);
      split2(v[2] * f, v[3] * f, h.y, l.y);
      split2(v[4] * f, v[5] * f, h.z, l.z);
      split2(v[6] * f, v[7] * f, h.w, l.w);
      // (columns past the matrix, up to the row stride, hold zeros)
      const long long at = ((long long)b * a.rows + r) * a.ldx + c;
      *(uint4*)(a.X[0][0] + at) = h;
      *(uint4*)(a.X[0][1] + at) = l;
    }
  }
}

// S from the gram partial tiles, summed in the order of the K ranges: a warp
// takes a 32 x 32 piece, lane = column.
__device__ __forceinline__ void join_gram(const OrthArgs& a, int warp, int nwarps) {
  const int lane = threadIdx.x & 31, nt = (a.m + BM - 1) / BM;
  const int items = a.batch * a.tiles * 16;
  const float f = 1.f / (1 << (2 * XE - SE));
  for (int it = warp; it < items; it += nwarps) {
    const int tile = it >> 4, rb = (it >> 2) & 3, cb = it & 3;
    const int b = tile / a.tiles;
    int i, j;
    triangle(tile - b * a.tiles, nt, i, j);
    const int row0 = i * BM + rb * 32, col = j * BM + cb * 32 + lane;
    if (row0 >= a.m || j * BM + cb * 32 >= a.m) continue;
    const float* p = a.part + (long long)tile * (BM * BM) + rb * 32 * BM + cb * 32 + lane;
    const long long step = (long long)a.batch * a.tiles * (BM * BM);
    float v[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) v[r] = 0.f;
    for (int k = 0; k < a.splits; ++k, p += step) {
#pragma unroll
      for (int r = 0; r < 32; ++r) v[r] += __ldcg(p + r * BM);
    }
#pragma unroll
    for (int r = 0; r < 32; ++r) v[r] *= f;
    if (col >= a.m) continue;
    const int nv = min(32, a.m - row0);
    const long long base = (long long)b * a.m * a.ldm;
    store_split_t(a.S[0] + base + row0 * a.ldm + col, a.S[1] + base + row0 * a.ldm + col, a.ldm, v,
                  nv);
    if (i != j)
      store_split(a.S[0] + base + col * a.ldm + row0, a.S[1] + base + col * a.ldm + row0, v, nv);
  }
}

__global__ void __launch_bounds__(THREADS, 1)
k_orth(const __grid_constant__ OrthMaps maps, const OrthArgs a) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = (uint64_t*)(smem + STAGES * STAGE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* done_bar = acc_empty + 2;
  uint32_t* tmem_holder = (uint32_t*)(done_bar + 1);
  volatile int* abort_flag = (volatile int*)(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&acc_full[s], 1);
      ptx::mbar_init(&acc_empty[s], 32 * EPI_WARPS);
    }
    ptx::mbar_init(done_bar, 1);
    ptx::fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_holder, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int phases_per_step = a.splits > 1 ? 4 : 3;  // gram, (join,) poly, update

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (ptx::elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      int issued[STAGES];
#pragma unroll
      for (int s = 0; s < STAGES; ++s) issued[s] = -1;
      for (int g = 0; g < 3 * a.steps && !*abort_flag; ++g) {
        const int step = g / 3, kind = g - 3 * step;
        const int ph = 1 + step * phases_per_step + (kind ? kind + phases_per_step - 3 : 0);
        const Work w = work_of(a, kind, step & 1);
        if (cta >= w.units) continue;
        if (!grid_wait(a, (unsigned)ph * ctas, abort_flag)) {
          give_up(a, abort_flag);
          break;
        }
        fence_proxy_async();
        for (int u = cta; u < w.units && !*abort_flag; u += ctas) {
          const Unit q = unit_of(a, w, u);
          for (int v = q.kb0 * w.terms; v < q.kb1 * w.terms; ++v) {
            const int kb = v / w.terms, term = v - kb * w.terms;
            if (!ptx::mbar_wait(&empty[stage], phase ^ 1, WAIT_NS)) {
              give_up(a, abort_flag);
              break;
            }
            ptx::mbar_arrive_expect_tx(&full[stage], A_BYTES + w.bn * BK * 2);
            unsigned char* sa = smem + stage * STAGE_BYTES;
            unsigned char* sb = sa + A_BYTES;
            const CUtensorMap* ma = &maps.m[w.a_buf][term == 2];
            const CUtensorMap* mb = &maps.m[w.b_buf][term == 1];
            // boxes of 64 x 64: K-major rows (k, row), MN-major rows (row, k)
#pragma unroll
            for (int j = 0; j < BM / 64; ++j) {
              const int r = q.m0 + 64 * j;
              tma_load_3d(sa + j * 8192, ma, &full[stage], w.a_mn ? r : kb * BK,
                          w.a_mn ? kb * BK : r, q.b);
            }
            for (int j = 0; j < w.bn / 64; ++j) {
              const int r = q.n0 + 64 * j;
              tma_load_3d(sb + j * 8192, mb, &full[stage], w.b_mn ? r : kb * BK,
                          w.b_mn ? kb * BK : r, q.b);
            }
#pragma unroll
            for (int s = 0; s < STAGES; ++s)
              if (s == stage) issued[s] = (int)phase;
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
          }
        }
      }
      // every load issued has landed before the block may end
#pragma unroll
      for (int s = 0; s < STAGES; ++s)
        if (issued[s] >= 0 && !ptx::mbar_wait(&full[s], (uint32_t)issued[s], WAIT_NS))
          give_up(a, abort_flag);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (ptx::elect_one()) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      for (int g = 0; g < 3 * a.steps && !*abort_flag; ++g) {
        const int step = g / 3, kind = g - 3 * step;
        const Work w = work_of(a, kind, step & 1);
        const uint32_t idesc = idesc_f16(w.bn, w.a_mn, w.b_mn);
        for (int u = cta; u < w.units && !*abort_flag; u += ctas) {
          const Unit q = unit_of(a, w, u);
          // (a block may wait here while others finish the product before: the
          // limit is that of its own loads, so this wait allows for theirs)
          if (!ptx::mbar_wait(&acc_empty[acc], acc_phase ^ 1, 4 * WAIT_NS)) {
            give_up(a, abort_flag);
            break;
          }
          ptx::tc_fence_after();
          const uint32_t d = tmem + acc * BN_MAX;
          bool ok = true;
          for (int v = q.kb0 * w.terms; v < q.kb1 * w.terms; ++v) {
            if (!ptx::mbar_wait(&full[stage], phase, 4 * WAIT_NS)) {
              give_up(a, abort_flag);
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const uint32_t a0 = ptx::smem_u32(smem + stage * STAGE_BYTES), b0 = a0 + A_BYTES;
            const int ksteps = min(BK / 16, (w.K - v / w.terms * BK + 15) / 16);
            for (int k = 0; k < ksteps; ++k) {
              const uint64_t ad = w.a_mn ? ptx::sdesc_sw128(a0 + k * 2048, 8192, 1024)
                                         : ptx::sdesc_sw128(a0 + k * 32, 16, 1024);
              const uint64_t bd = w.b_mn ? ptx::sdesc_sw128(b0 + k * 2048, 8192, 1024)
                                         : ptx::sdesc_sw128(b0 + k * 32, 16, 1024);
              ptx::mma_bf16(d, ad, bd, idesc, v > q.kb0 * w.terms || k > 0);
            }
            ptx::mma_commit(&empty[stage]);
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
          }
          if (!ok) break;
          ptx::mma_commit(&acc_full[acc]);
          if (++acc == 2) { acc = 0; acc_phase ^= 1; }
        }
      }
      // all issued MMAs complete before TMEM is released
      ptx::mma_commit(done_bar);
      if (!ptx::mbar_wait(done_bar, 0, WAIT_NS)) give_up(a, abort_flag);
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int et = threadIdx.x - 64, ew = et >> 5;
    const int sub = warp & 3, half = ew >> 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    unsigned ph = 0;
    // all of the block's writes of this phase, then one arrival for the block
    auto arrive = [&]() {
      fence_proxy_async();
      __threadfence();
      ptx::named_barrier(1, 32 * EPI_WARPS);
      if (et == 0) {
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.counter) : "memory");
      }
      ++ph;
    };
    auto wait = [&]() {
      const bool late = et == 0 && !grid_wait(a, ph * ctas, abort_flag);
      if (late) give_up(a, abort_flag);
      const bool ok = !epi_any(late);
      __threadfence();
      return ok;
    };
    if (a.in_f32) convert<float>(a, cta * 32 * EPI_WARPS + et, ctas * 32 * EPI_WARPS);
    else convert<__nv_bfloat16>(a, cta * 32 * EPI_WARPS + et, ctas * 32 * EPI_WARPS);
    arrive();
    bool ok = true;
    for (int g = 0; g < 3 * a.steps && ok; ++g) {
      const int step = g / 3, kind = g - 3 * step;
      const Work w = work_of(a, kind, step & 1);
      if (!(ok = wait())) break;
      for (int u = cta; u < w.units && ok; u += ctas) {
        const Unit q = unit_of(a, w, u);
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&acc_full[acc], acc_phase, 4 * WAIT_NS));
        if (!ok) {
          give_up(a, abort_flag);
          break;
        }
        ptx::tc_fence_after();
        const uint32_t t0 = tmem + acc * BN_MAX + ((uint32_t)(sub * 32) << 16);
        const int lrow = sub * 32 + lane;
#pragma unroll 1
        for (int c = half; c < w.bn / 32; c += 2) {
          float v[32];
          ptx::tmem_ld32(t0 + c * 32, v);
          ptx::tmem_ld_wait();
          ptx::reg_fence32(v);
          finish(a, w, q, step, step & 1, v, q.m0 + lrow, q.n0 + c * 32, lrow, c * 32);
          __syncwarp();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(&acc_empty[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      ok = !epi_any(!ok);
      if (!ok) break;
      arrive();
      if (kind == GRAM && a.splits > 1) {
        if (!(ok = wait())) break;
        join_gram(a, cta * EPI_WARPS + ew, ctas * EPI_WARPS);
        arrive();
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

// ---- host ------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (PFN_cuTensorMapEncodeTiled_v12000)f;
  });
  return fn;
}

// [batch][rows][ld] fp16, 64 x 64 boxes, 128-byte swizzle, zeros outside.
bool make_map(CUtensorMap* m, const void* p, long long rows, long long cols, long long ld,
              int batch) {
  auto fn = map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(rows * ld) * 2};
  const cuuint32_t box[3] = {64, 64, 1}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct OrthPlan {
  OrthArgs a;
  int ctas;
  size_t w_X[2][2], w_S[2], w_P[2], w_part, w_sums, w_sync, total;
};

constexpr int kSms = 152;  // (the plan may not depend on the device that runs it)

bool orth_plan(const rnnt_orth_dims* d, OrthPlan* p) {
  if (!d || d->rows < 1 || d->cols < 1 || d->batch < 0 || d->steps < 1 || d->steps > 32)
    return false;
  if (d->batch > 65535 || (long long)d->rows * d->cols > 2147483647LL || !(d->eps >= 0.f)) return false;
  if (!op_dtype(d->in_dtype) || !op_dtype(d->out_dtype)) return false;
  *p = OrthPlan{};
  OrthArgs& a = p->a;
  a.rows = d->rows; a.cols = d->cols; a.batch = d->batch; a.steps = d->steps; a.eps = d->eps;
  a.tall = a.rows > a.cols;
  a.m = a.tall ? a.cols : a.rows;
  a.n = a.tall ? a.rows : a.cols;
  a.in_f32 = d->in_dtype == RNNT_F32;
  a.out_f32 = d->out_dtype == RNNT_F32;
  a.in_ld = d->in_ld ? d->in_ld : a.cols;
  a.in_batch = d->in_batch ? d->in_batch : a.rows * a.in_ld;
  a.out_ld = d->out_ld ? d->out_ld : a.cols;
  a.out_batch = d->out_batch ? d->out_batch : a.rows * a.out_ld;
  if (a.in_ld < a.cols || a.out_ld < a.cols) return false;
  if (a.batch > 1 &&
      (a.in_batch < 0 || a.out_batch < (long long)(a.rows - 1) * a.out_ld + a.cols))
    return false;
  a.ldx = cdiv(a.cols, 8) * 8;
  a.ldm = cdiv(a.m, 8) * 8;
  const long long nt = cdiv(a.m, BM);
  a.tiles = (int)(nt * (nt + 1) / 2);
  // exact products where the result is fp32; for small matrices they cost
  // nothing (a product's time is its latency)
  a.terms = a.out_f32 || a.m <= 256 ? 3 : 1;
  // gram: K in as many ranges as there are SMs for its tiles, eight K blocks
  // at least (a range's partial tile costs as much as four)
  const int kbs = (int)cdiv(a.n, BK);
  const long long gu = (long long)a.batch * a.tiles;
  a.splits = (int)std::max<long long>(1, std::min<long long>(kSms / std::max(1LL, gu), kbs / 8));
  a.kb_split = (int)cdiv(kbs, a.splits);
  a.splits = (int)cdiv(kbs, a.kb_split);
  // update: 256-wide tiles when they fill the SMs
  const int un = a.tall ? a.m : a.n, um = a.tall ? a.n : a.m;
  a.ut_m = (int)cdiv(um, BM);
  a.bn = (long long)a.batch * a.ut_m * cdiv(un, 256) >= kSms ? 256 : 128;
  a.ut_n = (int)cdiv(un, a.bn);
  const long long units =
      std::max(gu * a.splits, (long long)a.batch * a.ut_m * a.ut_n);
  if ((long long)a.batch * a.ut_m * a.ut_n > 2147483647LL || gu * 16 > 2147483647LL) return false;
  p->ctas = (int)std::min<long long>(kSms, units);
  a.nb = (int)std::min<long long>(std::max<long long>(1, (long long)a.rows * a.cols / 4096), 256);
  const size_t x = 2 * (size_t)a.batch * a.rows * a.ldx, s = 2 * (size_t)a.batch * a.m * a.ldm;
  size_t o = 0;
  auto put = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes); return at; };
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) p->w_X[i][j] = put(x);
  for (int j = 0; j < 2; ++j) p->w_S[j] = put(s);
  for (int j = 0; j < 2; ++j) p->w_P[j] = put(s);
  p->w_part = put(a.splits > 1 ? 4 * (size_t)(gu * a.splits) * BM * BM : 0);
  p->w_sums = put(8 * (size_t)a.batch * a.nb);
  p->w_sync = put(8);
  p->total = o;
  return true;
}

cudaError_t orth_launch(OrthPlan& p, cudaStream_t st) {
  OrthArgs& a = p.a;
  OrthMaps maps;
  for (int j = 0; j < 2; ++j) {
    for (int i = 0; i < 2; ++i)
      if (!make_map(&maps.m[i][j], a.X[i][j], a.rows, a.cols, a.ldx, a.batch))
        return cudaErrorInvalidValue;
    if (!make_map(&maps.m[BUF_S][j], a.S[j], a.m, a.m, a.ldm, a.batch) ||
        !make_map(&maps.m[BUF_P][j], a.P[j], a.m, a.m, a.ldm, a.batch))
      return cudaErrorInvalidValue;
  }
  static std::atomic<bool> opted_in[kDeviceSlots];
  std::atomic<bool>& opted = opted_in[device_slot()];
  if (!opted.load()) {
    const cudaError_t e =
        cudaFuncSetAttribute(k_orth, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    opted.store(true);
  }
  double* sums = const_cast<double*>(a.sums);
  const dim3 grid(a.nb, a.batch);
  if (a.in_f32) k_orth_sumsq<float><<<grid, 256, 0, st>>>(a, sums);
  else k_orth_sumsq<__nv_bfloat16><<<grid, 256, 0, st>>>(a, sums);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // all blocks are resident at once (they wait for one another): cooperative
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  cfg.gridDim = dim3(std::min(p.ctas, num_sms()));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_orth, maps, a);
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
  OrthArgs& a = p.a;
  if (a.batch == 0) return RNNT_OK;
  if (!G || !O || !ws) return RNNT_ERR_INVALID_ARG;
  if (!aligned_to(G, op_size(dims->in_dtype)) || !aligned_to(O, op_size(dims->out_dtype)) ||
      !aligned_to(ws, ALIGN) || !aligned_to(status, 4))
    return RNNT_ERR_INVALID_ARG;
  if (ws_bytes < p.total) return RNNT_ERR_WORKSPACE_TOO_SMALL;
  char* w = (char*)ws;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) a.X[i][j] = (__half*)(w + p.w_X[i][j]);
  for (int j = 0; j < 2; ++j) {
    a.S[j] = (__half*)(w + p.w_S[j]);
    a.P[j] = (__half*)(w + p.w_P[j]);
  }
  a.part = (float*)(w + p.w_part);
  a.sums = (const double*)(w + p.w_sums);
  a.counter = (unsigned*)(w + p.w_sync);
  a.abort = (int*)(w + p.w_sync) + 1;
  a.G = G; a.O = O; a.status = status;
  cudaStream_t st = (cudaStream_t)stream;
  ProfScope ps("orth", st);
  ps.set_kernels(2);
  OPS_CHECK(orth_launch(p, st));
  return RNNT_OK;
}

}  // extern "C"
