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
//   exact (fp32 results, and small matrices, where it costs little): three
//     terms everywhere;
//   fast (bf16 results): one term in gram and update, whose rounding of 2^-12
//     per entry averages out over the row; three in poly, the smallest product,
//     because b S and c S S largely cancel near a singular value of 1.  For the
//     same reason P is taken off its mean there: for singular values near 1 its
//     diagonal is about d = b + c ... = -2.5, which the update applies in fp32
//     through (a + d) X.  The shift enters as the steps converge (it would cost
//     small singular values digits in the first ones).  In 64-bit emulation over
//     flat, 1/i^p and low-rank-plus-noise spectra the fast result is 0.3 to
//     1.6e-3 off, next to 1.7e-3 for its own rounding to bf16.  Up to five steps,
//     that is: small singular values grow by a a step, and their errors with them
//     (640 x 640, 1/i^2: 2.1e-3 off after five steps, 6.7e-3 after seven, 4.8e-2
//     after ten; exact 1.7, 1.7 and 1.9e-3).
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "../../include/rnnt_testing.h"
#include "ops.h"
#include "ptx.cuh"

namespace rnnt {
namespace {

// The Muon optimiser's quintic.
constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;

constexpr int BM = 128, BK = 64;      // tile rows; K per stage: a 128-byte swizzle atom of fp16
constexpr int BOX = 64 * 64 * 2;      // bytes of a TMA box
constexpr int RING = 192 * 1024, MAX_STAGES = 8;
constexpr int EPI_WARPS = 8, THREADS = 64 + 32 * EPI_WARPS + 32;
constexpr int PITCH = 80, STG = 32 * PITCH;  // an epilogue warp's staging rows of 64 bytes
constexpr int SMEM = 1024 + RING + EPI_WARPS * STG + 256;
// fast update: the ring ends here, and two 128 x 64 blocks of X (hi and lo) follow
constexpr int XBUF_AT = 144 * 1024, XPLANE = 128 * 128, XBUF = 2 * XPLANE;
static_assert(XBUF_AT + 2 * XBUF <= RING + EPI_WARPS * STG, "blocks of X lie in the ring and staging");
constexpr uint64_t WAIT_NS = 2000000000ull;  // per wait, then give up (2 s)
constexpr int XE = 14, SE = 14, PE = 13;     // scale exponents of X, S and P

enum { GRAM, POLY, UPDATE };

struct OrthMaps {  // X buffers 0 and 1, S, P; hi and lo of each
  CUtensorMap m[4][2];
};
enum { BUF_X0, BUF_X1, BUF_S, BUF_P };

struct OrthArgs {
  int m, n, tall, batch, steps;
  int exact;            // three terms in gram and update too
  int rows, cols;       // of G, and of X
  FastDiv chunks;       // of eight columns in a row
  long long ldx, ldm;   // row strides of X; of S and P
  __half* X[2][2];
  __half* S[2];
  __half* P[2];
  int thin;             // blocks per matrix of k_orth_thin (0: k_orth)
  float* part;          // gram partial tiles [splits][batch][tiles][128][bn];
                        // k_orth_thin: [batch][thin][128][128]
  float* sum;           // k_orth_thin: their sum [batch][128][128]
  int blocks;           // 128 x 128 blocks on and above the diagonal of S
  int splits, kb_split; // gram: K ranges and their length in K blocks
  int bn[3];            // tile width of each product
  int ut_m, ut_n;       // update: tiles
  int ut_whole;         // the tiles after these go out as two halves each
  const void* G;
  int in_f32;
  long long in_ld, in_batch;
  void* O;
  int out_f32;
  long long out_ld, out_batch;
  int out_vec;          // O takes 16-byte stores
  float eps;
  const double* sums;   // [batch][nb] partial sums of squares
  int nb;
  unsigned* counter;    // grid barriers: arrivals so far (one per matrix; k_orth has one)
  int* abort;
  int32_t* status;
  uint64_t wait_ns;
  int lost;             // 1: the first block never arrives at its first barrier (a test's)
};

// Eight consecutive elements of a row of G, those past nv 0.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int nv, bool vec, float (&v)[8]) {
  if (vec && nv >= 8) {
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
}

// ---- sums of squares ---------------------------------------------------------------
// Block (i, b) adds the squares of its share of matrix b: eight at a time in
// fp32, those in fp64.  A share whose squares left fp32's range, or whose sum is so
// small that squares below the range may count, is squared again in fp64 (in the
// first loop that would make 64 x 64 1.9 us longer, of 27; here it is 0.6).  Also
// clears the barrier of the kernel that follows.
__device__ __forceinline__ double block_sum(double s, double* part) {
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0;
  for (int k = 0; k < 8; ++k) s += part[k];
  return s;
}
template <typename T>
__global__ void __launch_bounds__(256)
k_orth_sumsq(OrthArgs a, double* sums) {
  __shared__ double part[8];
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.counter[blockIdx.y] = 0;
    if (blockIdx.y == 0) *a.abort = 0;
  }
  const T* g = (const T*)a.G + blockIdx.y * a.in_batch;
  const int chunks = a.chunks.d;
  const bool vec = a.in_ld % 8 == 0 && a.in_batch % 8 == 0 && ((uintptr_t)a.G & 15) == 0;
  double s = 0;
  // (unsigned: the last step may pass 2^31)
  const unsigned total = (unsigned)a.rows * chunks, stride = gridDim.x * 256;
  for (unsigned i0 = blockIdx.x * 256 + threadIdx.x; i0 < total; i0 += 4 * stride) {
    float v[4][8];  // four chunks' loads in flight
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const unsigned i = i0 + u * stride;
      const int r = (int)i / a.chunks, c = ((int)i - r * chunks) * 8;
      if (i < total) {
        load8<T>(g + r * a.in_ld + c, a.cols - c, vec, v[u]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u][k] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float q = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) q = fmaf(v[u][k], v[u][k], q);
      s += (double)q;
    }
  }
  s = block_sum(s, part);
  if (!(s > 1e-24 && s < 1e300)) {
    s = 0;
    for (unsigned i = blockIdx.x * 256 + threadIdx.x; i < total; i += stride) {
      float v[8];
      const int r = (int)i / a.chunks, c = ((int)i - r * chunks) * 8;
      load8<T>(g + r * a.in_ld + c, a.cols - c, vec, v);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (v[k] != 0.f) s = fma((double)v[k], (double)v[k], s);
    }
    s = block_sum(s, part);
  }
  if (threadIdx.x == 0) sums[blockIdx.y * (long long)gridDim.x + blockIdx.x] = s;
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
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, const void* src, int x, int y,
                                             int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(m),
      "r"(ptx::smem_u32(src)), "r"(x), "r"(y), "r"(z)
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

// One product: its tiles and operands.  fat: a stage holds hi and lo of both
// operands, and the two small terms add up in an accumulator of their own (the
// tensor cores' fp32 sums truncate: small terms added to a large sum would lose
// digits, and three adds per K step instead of one would truncate it more).
struct Work {
  int kind, units, kbs, K, bn, fat, a_mn, b_mn, a_buf, b_buf;
  int boxed;  // the epilogue's X comes and goes by TMA (fast update)
  int stage_bytes, stages;
};
struct Unit {
  int b, m0, n0, kb0, kb1, diag, bn;
};

template <int EXACT>
__device__ __forceinline__ Work work_of(const OrthArgs& a, int kind, int cur) {
  Work w;
  w.kind = kind;
  w.a_mn = w.b_mn = 0;
  w.bn = kind == GRAM ? a.bn[0] : kind == POLY ? a.bn[1] : a.bn[2];
  w.fat = EXACT;
  const int sym = a.batch * a.blocks * (BM / w.bn);
  if (kind == GRAM) {
    w.K = a.n;
    w.a_buf = w.b_buf = cur;
    w.a_mn = w.b_mn = a.tall;
    w.units = sym * a.splits;
  } else if (kind == POLY) {
    w.K = a.m;
    w.a_buf = w.b_buf = BUF_S;
    w.fat = 1;
    w.units = sym;
  } else {
    w.K = a.m;
    w.a_buf = a.tall ? cur : BUF_P;
    w.b_buf = a.tall ? BUF_P : cur;
    w.b_mn = !a.tall;
    w.units = 2 * a.batch * a.ut_m * a.ut_n - a.ut_whole;
  }
  w.kbs = (w.K + BK - 1) / BK;
  w.stage_bytes = (BM + w.bn) * BK * 2 << w.fat;
  w.boxed = !EXACT && kind == UPDATE;
  w.stages = min(MAX_STAGES, (w.boxed ? XBUF_AT : RING) / w.stage_bytes);
  return w;
}

__device__ __forceinline__ Unit unit_of(const OrthArgs& a, const Work& w, int u) {
  Unit q;
  q.kb0 = 0;
  q.kb1 = w.kbs;
  q.diag = 0;
  q.bn = w.bn;
  if (w.kind == UPDATE) {
    int t = u, right = 0;
    if (u >= a.ut_whole) {
      t = a.ut_whole + (u - a.ut_whole) / 2;
      right = (u - a.ut_whole) & 1;
      q.bn = w.bn / 2;
    }
    const int n = t % a.ut_n, rest = t / a.ut_n;
    q.b = rest / a.ut_m;
    q.m0 = (rest - q.b * a.ut_m) * BM;
    q.n0 = n * w.bn + right * q.bn;
    return q;
  }
  const int per_block = BM / w.bn, per = a.blocks * per_block;
  int rest = u;
  if (w.kind == GRAM && a.splits > 1) {
    const int ks = u / (a.batch * per);
    rest = u - ks * a.batch * per;
    q.kb0 = ks * a.kb_split;
    q.kb1 = min(w.kbs, q.kb0 + a.kb_split);
  }
  q.b = rest / per;
  rest -= q.b * per;
  int i, j;
  triangle(rest / per_block, (a.m + BM - 1) / BM, i, j);
  q.m0 = i * BM;
  q.n0 = j * BM + rest % per_block * w.bn;
  q.diag = i == j;
  return q;
}

// Wait until `target` blocks have arrived at the grid barrier in all.
__device__ __forceinline__ bool grid_wait(const OrthArgs& a, unsigned target,
                                          volatile int* abort_flag, int b = 0) {
  uint64_t t0 = 0;
  for (int i = 0;; ++i) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a.counter + b) : "memory");
    if (v >= target) return true;
    if ((i & 63) == 63) {
      if (*abort_flag || *(volatile int*)a.abort) return false;
      const uint64_t t = ptx::globaltimer();
      if (!t0) t0 = t;
      if (t - t0 > a.wait_ns) return false;
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

// ---- epilogue input and output ------------------------------------------------------
// A warp's 32 rows x 64 bytes of a row-major matrix, lane = row.  Global
// accesses take 8 rows x 64 bytes per instruction and pass through the warp's
// staging rows: one row per lane, 16 bytes of each, would touch 32 lines per
// instruction (that made the update's epilogue 12 us a tile, three times its
// products).  rows, bytes: how much of the block exists.
__device__ __forceinline__ void rows_issue(uint4 (&x)[4], const void* p, long long ld, int rows,
                                           int bytes) {
  const int lane = threadIdx.x & 31, piece = (lane & 3) * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    x[i] = r < rows && piece < bytes ? *(const uint4*)((const char*)p + r * ld + piece)
                                     : make_uint4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void rows_finish(unsigned char* stg, const uint4 (&x)[4],
                                            uint4 (&q)[4]) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *(uint4*)(stg + (i * 8 + (lane >> 2)) * PITCH + (lane & 3) * 16) = x[i];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = *(const uint4*)(stg + lane * PITCH + i * 16);
}
__device__ __forceinline__ void rows_store(unsigned char* stg, const uint4 (&q)[4], void* p,
                                           long long ld, int rows, int bytes) {
  const int lane = threadIdx.x & 31, piece = (lane & 3) * 16;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) *(uint4*)(stg + lane * PITCH + i * 16) = q[i];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    if (r < rows && piece < bytes)
      *(uint4*)((char*)p + r * ld + piece) = *(const uint4*)(stg + r * PITCH + piece);
  }
}

// 32 scaled values as 64 bytes of hi and of lo
__device__ __forceinline__ void split32(const float (&v)[32], uint4 (&h)[4], uint4 (&l)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    split2(v[8 * i], v[8 * i + 1], h[i].x, l[i].x);
    split2(v[8 * i + 2], v[8 * i + 3], h[i].y, l[i].y);
    split2(v[8 * i + 4], v[8 * i + 5], h[i].z, l[i].z);
    split2(v[8 * i + 6], v[8 * i + 7], h[i].w, l[i].w);
  }
}
__device__ __forceinline__ void add_halves(const uint4 (&q)[4], float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = unpack_h2(w[k]);
      v[8 * i + 2 * k] += x.x;
      v[8 * i + 2 * k + 1] += x.y;
    }
  }
}

// The transposed copy of a warp's block: value j of every lane goes to row j,
// at this lane's column (neighbouring lanes, neighbouring columns); nv rows
// exist, and this lane's column does.
__device__ __forceinline__ void store_t(__half* p, long long ld, const uint4 (&q)[4], int nv) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = 8 * i + 2 * k;
      if (j < nv) ((unsigned short*)p)[j * ld] = (unsigned short)w[k];
      if (j + 1 < nv) ((unsigned short*)p)[(j + 1) * ld] = (unsigned short)(w[k] >> 16);
    }
  }
}

// What the epilogue of a 32 x 32 block needs besides its products: S (poly) or
// X (update), asked for before the products are done.
struct Ahead {
  uint4 hi[4], lo[4];
};

struct Block {  // a warp's 32 x 32 block of a product
  int row0, col0, rows, cols;  // rows and columns of it that exist
};
__device__ __forceinline__ Block block_of(const OrthArgs& a, const Work& w, const Unit& q, int lrow0,
                                          int lcol0) {
  Block k;
  k.row0 = q.m0 + lrow0;
  k.col0 = q.n0 + lcol0;
  k.rows = (w.kind == UPDATE ? a.rows : a.m) - k.row0;
  k.cols = (w.kind == UPDATE ? a.cols : a.m) - k.col0;
  return k;
}

// (Planes' rows are padded to 16 bytes with zeros, which stay zeros: whole
// 16-byte pieces are read and written.)
__device__ __forceinline__ int plane_bytes(const Block& k) { return (k.cols + 7) / 8 * 16; }

__device__ __forceinline__ void look_ahead(const OrthArgs& a, const Work& w, const Unit& q, int cur,
                                           const Block& k, Ahead& h) {
  if (w.kind == GRAM) return;
  const __half *hi, *lo;
  long long ld, at;
  if (w.kind == UPDATE) {
    hi = a.X[cur][0]; lo = a.X[cur][1]; ld = a.ldx;
    at = ((long long)q.b * a.rows + k.row0) * ld + k.col0;
  } else {
    hi = a.S[0]; lo = a.S[1]; ld = a.ldm;
    at = ((long long)q.b * a.m + k.row0) * ld + k.col0;
  }
  rows_issue(h.hi, hi + at, ld * 2, k.rows, plane_bytes(k));
  rows_issue(h.lo, lo + at, ld * 2, k.rows, plane_bytes(k));
}

// v: the products of the block's row `lane`.
template <int EXACT>
__device__ __forceinline__ void finish(const OrthArgs& a, const Work& w, const Unit& q, int unit,
                                       int step, int cur, float (&v)[32], const Ahead& ahead,
                                       const Block& k, int lrow0, int lcol0, unsigned char* stg) {
  const int lane = threadIdx.x & 31;
  uint4 h[4], l[4];
  if (w.kind == GRAM && a.splits > 1) {
    float* p = a.part + ((long long)unit * BM + lrow0) * w.bn + lcol0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* x = v + 16 * half + 4 * i;
        h[i] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
      }
      rows_store(stg, h, p + 16 * half, w.bn * 4, 32, 64);
    }
    return;
  }
  if (k.rows <= 0 || k.cols <= 0) return;  // (the same for the whole warp)
  float x[32];
  if (w.kind != GRAM) {
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = 0.f;
    rows_finish(stg, ahead.hi, h);
    add_halves(h, x);
    rows_finish(stg, ahead.lo, h);
    add_halves(h, x);
  }
  if (EXACT && w.kind == UPDATE) {  // (fast: update_box)
    const float f = kA + shift_of(step);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = fmaf(f, x[j], v[j] * (1.f / (1 << PE)));
    if (step + 1 < a.steps) {
      const long long at = ((long long)q.b * a.rows + k.row0) * a.ldx + k.col0;
      split32(v, h, l);
      rows_store(stg, h, a.X[cur ^ 1][0] + at, a.ldx * 2, k.rows, plane_bytes(k));
      rows_store(stg, l, a.X[cur ^ 1][1] + at, a.ldx * 2, k.rows, plane_bytes(k));
      return;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= 1.f / (1 << XE);
    const long long o = q.b * a.out_batch + k.row0 * a.out_ld + k.col0;
    if (!a.out_vec) {
      if (lane >= k.rows) return;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (j >= k.cols) continue;
        if (a.out_f32) ((float*)a.O)[o + lane * a.out_ld + j] = v[j];
        else ((__nv_bfloat16*)a.O)[o + lane * a.out_ld + j] = __float2bfloat16_rn(v[j]);
      }
    } else if (a.out_f32) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* y = v + 16 * half + 4 * i;
          h[i] = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                            __float_as_uint(y[3]));
        }
        rows_store(stg, h, (float*)a.O + o + 16 * half, a.out_ld * 4, k.rows,
                   (k.cols - 16 * half) * 4);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* y = v + 8 * i;
        h[i] = make_uint4(ptx::pack_bf16x2(y[0], y[1]), ptx::pack_bf16x2(y[2], y[3]),
                          ptx::pack_bf16x2(y[4], y[5]), ptx::pack_bf16x2(y[6], y[7]));
      }
      rows_store(stg, h, (__nv_bfloat16*)a.O + o, a.out_ld * 2, k.rows, k.cols * 2);
    }
    return;
  }
  __half* const* out = a.S;
  bool lo = true;
  if (w.kind == GRAM) {
    const float f = 1.f / (1 << (2 * XE - SE));
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= f;
  } else {
    const float fs = kB / (1 << (SE - PE)), fp = kC / (1 << (2 * SE - PE));
    const float d = shift_of(step) * (1 << PE);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      v[j] = fmaf(fs, x[j], v[j] * fp) - (k.row0 + lane == k.col0 + j ? d : 0.f);
    out = a.P;
    lo = EXACT;  // (the update's one term takes P's hi alone)
  }
  split32(v, h, l);
  const long long base = (long long)q.b * a.m * a.ldm, at = base + k.row0 * a.ldm + k.col0;
  const long long t = base + k.col0 * a.ldm + k.row0 + lane;
  rows_store(stg, h, out[0] + at, a.ldm * 2, k.rows, plane_bytes(k));
  if (!q.diag && lane < k.rows) store_t(out[0] + t, a.ldm, h, k.cols);
  if (!lo) return;
  rows_store(stg, l, out[1] + at, a.ldm * 2, k.rows, plane_bytes(k));
  if (!q.diag && lane < k.rows) store_t(out[1] + t, a.ldm, l, k.cols);
}

// Blocks of 64 columns of a fast update's tile.
__device__ __forceinline__ int boxes_of(const OrthArgs& a, const Unit& q) {
  return min(q.bn / 64, (a.cols - q.n0 + 63) / 64);
}

// Fast update of 32 columns of the thread's row of an X block in shared memory
// (128-byte swizzled rows, hi and lo planes): x <- f x + v in place; after the
// last step the result to O, through the hi plane.
__device__ __forceinline__ void update_box(const OrthArgs& a, const Unit& q, int step,
                                           float (&v)[32], unsigned char* p, int row, int col,
                                           int out_col) {
  const float f = kA + shift_of(step);
  uint4 h[4], l[4];
  const uint32_t r0 = row * 128, sw = row & 7, c0 = col >> 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = *(const uint4*)(p + r0 + (((c0 + i) ^ sw) << 4));
    l[i] = *(const uint4*)(p + XPLANE + r0 + (((c0 + i) ^ sw) << 4));
  }
  float x[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) x[j] = 0.f;
  add_halves(h, x);
  add_halves(l, x);
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = fmaf(f, x[j], v[j] * (1.f / (1 << PE)));
  if (step + 1 < a.steps) {
    split32(v, h, l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *(uint4*)(p + r0 + (((c0 + i) ^ sw) << 4)) = h[i];
      *(uint4*)(p + XPLANE + r0 + (((c0 + i) ^ sw) << 4)) = l[i];
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] *= 1.f / (1 << XE);
  __nv_bfloat16* o = (__nv_bfloat16*)a.O + q.b * a.out_batch;
  const int cols = a.cols - out_col, lane = threadIdx.x & 31;
  if (!a.out_vec) {
    if (q.m0 + row >= a.rows) return;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < cols) o[(q.m0 + row) * a.out_ld + out_col + j] = __float2bfloat16_rn(v[j]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *(uint4*)(p + r0 + (((c0 + i) ^ sw) << 4)) = make_uint4(
        ptx::pack_bf16x2(v[8 * i], v[8 * i + 1]), ptx::pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
        ptx::pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), ptx::pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (row & ~31) + i * 8 + (lane >> 2), piece = lane & 3;
    if (q.m0 + r < a.rows && 8 * piece < cols)
      *(uint4*)(o + (q.m0 + r) * a.out_ld + out_col + 8 * piece) =
          *(const uint4*)(p + r * 128 + (((c0 + piece) ^ (r & 7)) << 4));
  }
}

// 1 / (|G|_F + eps) of matrix b in two factors, the same in every lane: pre, a power
// of two that brings norms outside 2^-100 to 2^100 back (1 for all others), and f
// (0 for a matrix of zeros, NaN when the norm is not finite).
struct Scale {
  float pre, f;
};
__device__ __forceinline__ Scale inverse_norm(const OrthArgs& a, int b) {
  const int lane = threadIdx.x & 31;
  double s = 0;
  for (int i = lane; i < a.nb; i += 32) s += a.sums[(long long)b * a.nb + i];
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (!isfinite(s)) return {1.f, __int_as_float(0x7fc00000)};
  // square root in fp32 of the sum scaled by an even power of two (fp64 square
  // roots and divisions take microseconds here)
  if (!(s > 0)) return {1.f, 0.f};
  const int e = (((int)(__double2hiint(s) >> 20) & 0x7ff) - 1023) & ~1;
  const int up = e / 2 > 100 ? -60 : e / 2 < -100 ? 60 : 0;
  const float pre = up < 0 ? 0x1p-60f : up > 0 ? 0x1p60f : 1.f;
  const float r = ldexpf(sqrtf((float)(s * __hiloint2double((1023 - e) << 20, 0))), e / 2 + up);
  return {pre, 1.f / (r + a.eps * pre)};
}

// X = G / (|G|_F + eps) as hi and lo planes (epilogue warps of all blocks), four
// chunks of eight in flight.
template <typename T>
__device__ __forceinline__ void convert(const OrthArgs& a, int tid, int nthreads) {
  const int chunks = a.chunks.d;
  const unsigned per = (unsigned)a.rows * chunks;
  const bool vec = a.in_ld % 8 == 0 && a.in_batch % 8 == 0 && ((uintptr_t)a.G & 15) == 0;
  for (int b = 0; b < a.batch; ++b) {
    const Scale sc = inverse_norm(a, b);
    const float pre = sc.pre, f = sc.f * (1 << XE);
    for (unsigned i0 = tid; i0 < per; i0 += 4 * nthreads) {
      float v[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const unsigned i = i0 + u * nthreads;
        const int r = (int)i / a.chunks, c = ((int)i - r * chunks) * 8;
        if (i < per)
          load8<T>((const T*)a.G + b * a.in_batch + r * a.in_ld + c, a.cols - c, vec, v[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const unsigned i = i0 + u * nthreads;
        if (i >= per) break;
        const int r = (int)i / a.chunks, c = ((int)i - r * chunks) * 8;
        uint4 h, l;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u][k] *= pre;
        split2(v[u][0] * f, v[u][1] * f, h.x, l.x);
        split2(v[u][2] * f, v[u][3] * f, h.y, l.y);
        split2(v[u][4] * f, v[u][5] * f, h.z, l.z);
        split2(v[u][6] * f, v[u][7] * f, h.w, l.w);
        // (columns past the matrix, up to the row stride, hold zeros)
        const long long at = ((long long)b * a.rows + r) * a.ldx + c;
        *(uint4*)(a.X[0][0] + at) = h;
        *(uint4*)(a.X[0][1] + at) = l;
      }
    }
  }
}

// S from the gram partial tiles, summed in the order of the K ranges: a warp
// takes 8 rows x 32 columns, lane = column, four ranges' loads in flight.
__device__ __forceinline__ void join_gram(const OrthArgs& a, int warp, int nwarps) {
  const int lane = threadIdx.x & 31, nt = (a.m + BM - 1) / BM, bn = a.bn[0];
  const int per_block = BM / bn, per_unit = 16 * (bn / 32);
  const int units = a.batch * a.blocks * per_block;
  const float f = 1.f / (1 << (2 * XE - SE));
  const long long step = (long long)units * BM * bn;
  for (int it = warp; it < units * per_unit; it += nwarps) {
    const int unit = it / per_unit, piece = it - unit * per_unit;
    const int rg = piece & 15, cb = piece >> 4;
    const int b = unit / (a.blocks * per_block), rest = unit - b * a.blocks * per_block;
    int i, j;
    triangle(rest / per_block, nt, i, j);
    const int row0 = i * BM + rg * 8, colb = j * BM + rest % per_block * bn + cb * 32;
    const int col = colb + lane;
    if (row0 >= a.m || colb >= a.m) continue;
    const float* p = a.part + ((long long)unit * BM + rg * 8) * bn + cb * 32 + lane;
    float v[8] = {};
    int k = 0;
    for (; k + 4 <= a.splits; k += 4, p += 4 * step) {
      float x[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int r = 0; r < 8; ++r) x[u][r] = __ldcg(p + u * step + r * bn);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] += x[u][r];
    }
    for (; k < a.splits; ++k, p += step) {
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] += __ldcg(p + r * bn);
    }
    if (col >= a.ldm) continue;
    uint4 h, l;
    split2(v[0] * f, v[1] * f, h.x, l.x);
    split2(v[2] * f, v[3] * f, h.y, l.y);
    split2(v[4] * f, v[5] * f, h.z, l.z);
    split2(v[6] * f, v[7] * f, h.w, l.w);
    const long long base = (long long)b * a.m * a.ldm;
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if (row0 + r >= a.m) break;
      const long long at = base + (row0 + r) * a.ldm + col;
      ((unsigned short*)a.S[0])[at] = (unsigned short)(hw[r / 2] >> (16 * (r & 1)));
      ((unsigned short*)a.S[1])[at] = (unsigned short)(lw[r / 2] >> (16 * (r & 1)));
    }
    if (i != j && col < a.m) {  // (the eight rows, past m zeros, are one 16-byte piece)
      const long long at = base + col * a.ldm + row0;
      *(uint4*)(a.S[0] + at) = h;
      *(uint4*)(a.S[1] + at) = l;
    }
  }
}

template <int EXACT>
__global__ void __launch_bounds__(THREADS, 1)
k_orth(const __grid_constant__ OrthMaps maps, const OrthArgs a) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char* staging = smem + RING;
  uint64_t* full = (uint64_t*)(staging + EPI_WARPS * STG);
  uint64_t* empty = full + MAX_STAGES;
  uint64_t* acc_full = empty + MAX_STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* x_full = acc_empty + 2;  // X blocks: loaded, done with, all stored
  uint64_t* x_done = x_full + 2;
  uint64_t* x_stored = x_done + 2;
  uint64_t* done_bar = x_stored + 1;
  uint32_t* tmem_holder = (uint32_t*)(done_bar + 1);
  volatile int* abort_flag = (volatile int*)(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&acc_full[s], 1);
      ptx::mbar_init(&acc_empty[s], 32 * EPI_WARPS);
      ptx::mbar_init(&x_full[s], 1);
      ptx::mbar_init(&x_done[s], EPI_WARPS);
    }
    ptx::mbar_init(x_stored, 1);
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
  // Every product lays its own stages over the ring, from stage 0 on (the grid
  // barrier before it says that the ring is idle); `par` has each stage
  // barrier's parity.
  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (ptx::elect_one()) {
      uint32_t par = 0, used = 0;
      for (int g = 0; g < 3 * a.steps && !*abort_flag; ++g) {
        const int step = g / 3, kind = g - 3 * step;
        const int ph = 1 + step * phases_per_step + (kind ? kind + phases_per_step - 3 : 0);
        const Work w = work_of<EXACT>(a, kind, step & 1);
        if (cta >= w.units) continue;
        if (!grid_wait(a, (unsigned)ph * ctas, abort_flag)) {
          give_up(a, abort_flag);
          break;
        }
        fence_proxy_async();
        int stage = 0;
        for (int u = cta; u < w.units && !*abort_flag; u += ctas) {
          const Unit q = unit_of(a, w, u);
          for (int kb = q.kb0; kb < q.kb1; ++kb) {
            if (!ptx::mbar_wait(&empty[stage], (par >> stage & 1) ^ 1, a.wait_ns)) {
              give_up(a, abort_flag);
              break;
            }
            // (a block on the diagonal multiplies its rows by themselves: one load)
            ptx::mbar_arrive_expect_tx(&full[stage],
                                       (BM + (q.diag ? 0 : q.bn)) * BK * 2 << w.fat);
            unsigned char* d = smem + stage * w.stage_bytes;
            // boxes of 64 x 64: K-major rows (k, row), MN-major rows (row, k)
            const int k0 = kb * BK;
            for (int pl = 0; pl <= w.fat; ++pl, d += 2 * BOX) {
              const CUtensorMap* m = &maps.m[w.a_buf][pl];
              tma_load_3d(d, m, &full[stage], w.a_mn ? q.m0 : k0, w.a_mn ? k0 : q.m0, q.b);
              tma_load_3d(d + BOX, m, &full[stage], w.a_mn ? q.m0 + 64 : k0,
                          w.a_mn ? k0 : q.m0 + 64, q.b);
            }
            for (int pl = 0; pl <= w.fat && !q.diag; ++pl) {
              const CUtensorMap* m = &maps.m[w.b_buf][pl];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (64 * j >= q.bn) break;
                const int r = q.n0 + 64 * j;
                tma_load_3d(d, m, &full[stage], w.b_mn ? r : k0, w.b_mn ? k0 : r, q.b);
                d += BOX;
              }
            }
            par ^= 1u << stage;
            used |= 1u << stage;
            if (++stage == w.stages) stage = 0;
          }
        }
      }
      // every load issued has landed before the block may end
      for (int s = 0; s < MAX_STAGES; ++s)
        if (used >> s & 1 && !ptx::mbar_wait(&full[s], (par >> s & 1) ^ 1, a.wait_ns))
          give_up(a, abort_flag);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (ptx::elect_one()) {
      uint32_t par = 0, acc_phase = 0;
      int acc = 0;
      for (int g = 0; g < 3 * a.steps && !*abort_flag; ++g) {
        const int step = g / 3, kind = g - 3 * step;
        const Work w = work_of<EXACT>(a, kind, step & 1);
        // 16-byte units: planes, one K step of 16 in each layout, and the
        // descriptors without their address
        const uint32_t plane_a = BM * BK * 2 / 16;
        const uint32_t step_a = w.a_mn ? 128 : 2, step_b = w.b_mn ? 128 : 2;
        const uint64_t desc_a = ptx::sdesc_sw128(0, w.a_mn ? 8192 : 16, 1024);
        const uint64_t desc_b = ptx::sdesc_sw128(0, w.b_mn ? 8192 : 16, 1024);
        const uint32_t smem_a = ptx::smem_u32(smem);
        int stage = 0;
        for (int u = cta; u < w.units && !*abort_flag; u += ctas) {
          const Unit q = unit_of(a, w, u);
          // (these waits allow for the other blocks' products before as well)
          if (!ptx::mbar_wait(&acc_empty[acc], acc_phase ^ 1, 4 * a.wait_ns)) {
            give_up(a, abort_flag);
            break;
          }
          ptx::tc_fence_after();
          const uint32_t d = tmem + acc * 256, idesc = idesc_f16(q.bn, w.a_mn, w.b_mn);
          const uint32_t plane_b = q.bn * BK * 2 / 16;
          bool ok = true;
          for (int kb = q.kb0; kb < q.kb1; ++kb) {
            if (!ptx::mbar_wait(&full[stage], par >> stage & 1, 4 * a.wait_ns)) {
              give_up(a, abort_flag);
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            // (one thread issues every MMA: descriptors are stepped, not built)
            const uint64_t sa = (smem_a + stage * w.stage_bytes) >> 4;
            const uint64_t ah = desc_a + sa, al = ah + plane_a;
            const uint64_t bh = desc_b + sa + (q.diag ? (q.n0 - q.m0) * (BK * 2 / 16)
                                                      : plane_a << w.fat);
            const uint64_t bl = bh + (q.diag ? plane_a : plane_b);
            const int ksteps = min(BK / 16, (w.K - kb * BK + 15) / 16);
            uint32_t more = kb > q.kb0;
            if (EXACT || w.fat) {
#pragma unroll
              for (int k = 0; k < BK / 16; ++k) {
                if (k >= ksteps) break;
                const uint64_t ka = k * step_a, kb_ = k * step_b;
                ptx::mma_bf16(d, ah + ka, bh + kb_, idesc, more);
                ptx::mma_bf16(d + 128, ah + ka, bl + kb_, idesc, more);
                ptx::mma_bf16(d + 128, al + ka, bh + kb_, idesc, 1);
                more = 1;
              }
            } else {
#pragma unroll
              for (int k = 0; k < BK / 16; ++k) {
                if (k >= ksteps) break;
                ptx::mma_bf16(d, ah + k * step_a, bh + k * step_b, idesc, more);
                more = 1;
              }
            }
            ptx::mma_commit(&empty[stage]);
            par ^= 1u << stage;
            if (++stage == w.stages) stage = 0;
          }
          if (!ok) break;
          ptx::mma_commit(&acc_full[acc]);
          if (++acc == 2) { acc = 0; acc_phase ^= 1; }
        }
      }
      // all issued MMAs complete before TMEM is released
      ptx::mma_commit(done_bar);
      if (!ptx::mbar_wait(done_bar, 0, a.wait_ns)) give_up(a, abort_flag);
    }
  } else if (warp == 2 + EPI_WARPS) {
    // ---------------------------------------------------------------- X blocks
    // Fast update: loads the 128 x 64 blocks of X (hi and lo) that the epilogue
    // updates in place, two at a time, and stores them to the other X.
    if (!EXACT && ptx::elect_one()) {
      unsigned char* xbuf = smem + XBUF_AT;
      int n_load = 0, n_done = 0;
      bool ok = true;
      for (int step = 0; step < a.steps && ok; ++step) {
        const int cur = step & 1;
        const Work w = work_of<EXACT>(a, UPDATE, cur);
        if (cta >= w.units) continue;
        if (!grid_wait(a, (unsigned)((step + 1) * phases_per_step) * ctas, abort_flag)) {
          give_up(a, abort_flag);
          break;
        }
        fence_proxy_async();
        const bool last = step + 1 == a.steps;
        // two walks over the same blocks: the loads run two ahead of the stores
        int lu = cta, lc = 0, su = cta, sc = 0;
        while (ok && su < w.units) {
          while (lu < w.units && n_load < n_done + 2) {
            const Unit q = unit_of(a, w, lu);
            unsigned char* d = xbuf + (n_load & 1) * XBUF;
            uint64_t* bar = &x_full[n_load & 1];
            ptx::mbar_arrive_expect_tx(bar, XBUF);
#pragma unroll
            for (int j = 0; j < 4; ++j)  // hi rows 0-63, 64-127, lo rows 0-63, 64-127
              tma_load_3d(d + j * BOX, &maps.m[cur][j >> 1], bar, q.n0 + 64 * lc,
                          q.m0 + 64 * (j & 1), q.b);
            ++n_load;
            if (++lc == boxes_of(a, q)) { lc = 0; lu += ctas; }
          }
          const Unit q = unit_of(a, w, su);
          if (!ptx::mbar_wait(&x_done[n_done & 1], n_done >> 1 & 1, 4 * a.wait_ns)) {
            give_up(a, abort_flag);
            ok = false;
            break;
          }
          if (!last) {
            const unsigned char* d = xbuf + (n_done & 1) * XBUF;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (q.m0 + 64 * (j & 1) < a.rows)
                tma_store_3d(&maps.m[cur ^ 1][j >> 1], d + j * BOX, q.n0 + 64 * sc,
                             q.m0 + 64 * (j & 1), q.b);
            ptx::bulk_commit();
            ptx::bulk_wait_read();
          }
          ++n_done;
          if (++sc == boxes_of(a, q)) { sc = 0; su += ctas; }
        }
        ptx::bulk_wait_all();
        ptx::mbar_arrive(x_stored);
      }
      // every load issued has landed before the block may end
      for (int i = n_done; i < n_load; ++i)
        if (!ptx::mbar_wait(&x_full[i & 1], i >> 1 & 1, a.wait_ns)) give_up(a, abort_flag);
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int et = threadIdx.x - 64, ew = et >> 5;
    const int sub = warp & 3, half = ew >> 2;
    unsigned char* stg = staging + ew * STG;
    int acc = 0, n_box = 0;
    uint32_t acc_phase = 0;
    unsigned ph = 0;
    // One arrival for the block, after all of its writes of this phase (the
    // barrier orders the other threads' writes before thread 0's release, which
    // is fence enough: one more made a phase 0.4 us longer).
    auto arrive = [&]() {
      ptx::named_barrier(1, 32 * EPI_WARPS);
      if (et == 0 && !(a.lost && cta == 0 && ph == 0))
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.counter) : "memory");
      ++ph;
    };
    auto wait = [&]() {
      const bool late = et == 0 && !grid_wait(a, ph * ctas, abort_flag);
      if (late) give_up(a, abort_flag);
      return !epi_any(late);
    };
    if (a.in_f32) convert<float>(a, cta * 32 * EPI_WARPS + et, ctas * 32 * EPI_WARPS);
    else convert<__nv_bfloat16>(a, cta * 32 * EPI_WARPS + et, ctas * 32 * EPI_WARPS);
    arrive();
    bool ok = true;
    for (int g = 0; g < 3 * a.steps && ok; ++g) {
      const int step = g / 3, kind = g - 3 * step;
      const Work w = work_of<EXACT>(a, kind, step & 1);
      if (!(ok = wait())) break;
      for (int u = cta; u < w.units && ok; u += ctas) {
        const Unit q = unit_of(a, w, u);
        Ahead ahead;
        Block k = block_of(a, w, q, sub * 32, half * 32);
        if (!w.boxed) look_ahead(a, w, q, step & 1, k, ahead);
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&acc_full[acc], acc_phase, 4 * a.wait_ns));
        if (!ok) {
          give_up(a, abort_flag);
          break;
        }
        ptx::tc_fence_after();
        const uint32_t t0 = tmem + acc * 256 + ((uint32_t)(sub * 32) << 16);
        if (!EXACT && w.boxed) {
          const int boxes = boxes_of(a, q);
#pragma unroll 1
          for (int c = 0; c < boxes; ++c, ++n_box) {
            float v[32];
            ptx::tmem_ld32(t0 + c * 64 + half * 32, v);
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&x_full[n_box & 1], n_box >> 1 & 1,
                                                        4 * a.wait_ns));
            ptx::tmem_ld_wait();
            ptx::reg_fence32(v);
            if (!ok) {
              give_up(a, abort_flag);
              break;
            }
            update_box(a, q, step, v, smem + XBUF_AT + (n_box & 1) * XBUF, sub * 32 + lane,
                       half * 32, q.n0 + c * 64 + half * 32);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&x_done[n_box & 1]);
            __syncwarp();
          }
          if (!ok) break;
          ptx::tc_fence_before();
          ptx::mbar_arrive(&acc_empty[acc]);
          if (++acc == 2) { acc = 0; acc_phase ^= 1; }
          continue;
        }
#pragma unroll 1
        for (int c = half; c < q.bn / 32; c += 2) {
          float v[32];
          ptx::tmem_ld32(t0 + c * 32, v);
          if (EXACT || w.fat) {
            float x[32];
            ptx::tmem_ld32(t0 + 128 + c * 32, x);
            ptx::tmem_ld_wait();
            ptx::reg_fence32(v);
            ptx::reg_fence32(x);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += x[j];
          } else {
            ptx::tmem_ld_wait();
            ptx::reg_fence32(v);
          }
          const Ahead now = ahead;
          const Block kn = k;
          if (c + 2 < q.bn / 32) {
            k = block_of(a, w, q, sub * 32, (c + 2) * 32);
            look_ahead(a, w, q, step & 1, k, ahead);
          }
          finish<EXACT>(a, w, q, u, step, step & 1, v, now, kn, sub * 32, c * 32, stg);
          __syncwarp();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(&acc_empty[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      // (the X blocks are stored by another warp)
      if (!EXACT && w.boxed && cta < w.units && ok && et == 0)
        ok = ptx::mbar_wait(x_stored, step & 1, 4 * a.wait_ns);
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
  __syncwarp();  // (of the first warps one lane alone worked)
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

// ---- thin matrices --------------------------------------------------------------------
// m <= 128: everything stays on chip.  A block keeps 128 columns of X (rows of a
// tall one, transposed on the way in and out) as hi and lo in shared memory, in
// the swizzled layout that serves both as the K-major operand of its share of
// S and as the MN-major operand of its share of P X; S, then P over it, have the
// same layout.  So a product is three MMA chains and a pass of the 128 x 128
// accumulator through registers, about 0.7 us, against 4.4 us through global
// memory and a grid barrier; only the blocks' shares of S meet, once per step:
// over the shared memory of a cluster for up to 16 blocks (128 x 2048: 91 us,
// 126 x 142: 72), else through global memory (132 and 107).  All products exact.
constexpr int THIN_THREADS = 256;
constexpr int IMG = 128 * 128 * 2;           // bytes of a 128 x 128 plane: two 64-column blocks
constexpr int THIN_SMEM = 1024 + 4 * IMG + 256;
// A cluster's blocks take their pieces of S here: 8 rows x 64 columns in fp32, 32
// at most, dealt out evenly, each from every block (at most 45 for 2 to 16 blocks).
constexpr int MAX_THIN_CLUSTER = 16, PIECE = 8 * 64 * 4;
constexpr int THIN_CLUSTER_SMEM = THIN_SMEM + 45 * PIECE;

// byte of (row, col) in a plane, col a multiple of 8
__device__ __forceinline__ uint32_t img_at(int row, int col) {
  return (col >> 6) * (IMG / 2) + row * 128 + (((col >> 3 & 7) ^ (row & 7)) << 4);
}

// v of (row, col0 .. col0 + 31) as hi and lo, to or from the planes at p
__device__ __forceinline__ void img_store(unsigned char* p, int row, int col0,
                                          const float (&v)[32]) {
  uint4 h[4], l[4];
  split32(v, h, l);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t at = img_at(row, col0 + 8 * i);
    *(uint4*)(p + at) = h[i];
    *(uint4*)(p + IMG + at) = l[i];
  }
}
__device__ __forceinline__ void img_load(const unsigned char* p, int row, int col0,
                                         float (&v)[32]) {
  uint4 h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t at = img_at(row, col0 + 8 * i);
    h[i] = *(const uint4*)(p + at);
    l[i] = *(const uint4*)(p + IMG + at);
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = 0.f;
  add_halves(h, v);
  add_halves(l, v);
}

// The block's columns j0 .. of X into the planes at p (zeros outside).
template <typename T>
__device__ __forceinline__ void thin_load(const OrthArgs& a, int b, int j0, unsigned char* p) {
  const T* g = (const T*)a.G + b * a.in_batch;
  const bool vec = a.in_ld % 8 == 0 && a.in_batch % 8 == 0 && ((uintptr_t)a.G & 15) == 0;
  const Scale sc = inverse_norm(a, b);
  const float pre = sc.pre, f = sc.f * (1 << XE);
  for (int t = threadIdx.x; t < 128 * 16; t += THIN_THREADS) {
    // eight neighbours in memory: columns of a row of X, or (tall) rows of a column
    const int line = t >> 4, c = (t & 15) * 8;
    const int lines = a.tall ? a.n - j0 : a.m, left = (a.tall ? a.m : a.n - j0) - c;
    float v[8] = {};
    if (line < lines && left > 0)
      load8<T>(a.tall ? g + (j0 + line) * a.in_ld + c : g + line * a.in_ld + j0 + c, left, vec, v);
    uint4 h, l;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= pre;
    split2(v[0] * f, v[1] * f, h.x, l.x);
    split2(v[2] * f, v[3] * f, h.y, l.y);
    split2(v[4] * f, v[5] * f, h.z, l.z);
    split2(v[6] * f, v[7] * f, h.w, l.w);
    if (!a.tall) {
      const uint32_t at = img_at(line, c);
      *(uint4*)(p + at) = h;
      *(uint4*)(p + IMG + at) = l;
    } else {
      const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t at = img_at(c + k, line & ~7) + (line & 7) * 2;
        *(unsigned short*)(p + at) = (unsigned short)(hw[k / 2] >> (16 * (k & 1)));
        *(unsigned short*)(p + IMG + at) = (unsigned short)(lw[k / 2] >> (16 * (k & 1)));
      }
    }
  }
}

// D += A B^T over `ksteps` steps of 16, three terms: hi hi at d, the small ones
// at d + 128.  A K-major at pa; B K-major or MN-major (b_mn) at pb.
__device__ __forceinline__ void thin_mma(uint32_t d, uint32_t pa, uint32_t pb, int b_mn, int n,
                                         int ksteps) {
  const uint32_t idesc = idesc_f16(n, 0, b_mn);
  // (one thread issues them: the descriptors are stepped, in 16-byte units)
  const uint64_t da = ptx::sdesc_sw128(pa, 16, 1024);
  const uint64_t db = ptx::sdesc_sw128(pb, b_mn ? IMG / 2 : 16, 1024);
  constexpr uint32_t LO = IMG / 16, BLOCK = IMG / 32;
  uint32_t more = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k >= ksteps) break;
    const uint32_t ko = (k >> 2) * BLOCK + (k & 3) * 2, kb = b_mn ? k * 128 : ko;
    ptx::mma_bf16(d, da + ko, db + kb, idesc, more);
    ptx::mma_bf16(d + 128, da + ko, db + kb + LO, idesc, more);
    ptx::mma_bf16(d + 128, da + ko + LO, db + kb, idesc, 1);
    more = 1;
  }
}

// The blocks' shares of S, summed: block c of `blocks` adds slice c of all
// shares [blocks][m][128], in order of the blocks (eight ranges of them, one
// per warp, when there are many).
__device__ __forceinline__ void thin_reduce(const float* part, float* sum, int c, int blocks, int m,
                                            float4 (*tmp)[32]) {
  const int groups = m * 32, per = (groups + blocks - 1) / blocks;
  const int g0 = c * per, g1 = min(groups, g0 + per);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float4* p = (const float4*)part;
  auto add = [](float4& s, const float4& x) {
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  };
  if (blocks < 16) {
    for (int g = g0 + threadIdx.x; g < g1; g += THIN_THREADS) {
      float4 s = make_float4(0, 0, 0, 0);
#pragma unroll 4
      for (int k = 0; k < blocks; ++k) add(s, __ldcg(p + (long long)k * 4096 + g));
      ((float4*)sum)[g] = s;
    }
    return;
  }
  const int range = (blocks + 7) / 8, k0 = warp * range, k1 = min(blocks, k0 + range);
  for (int gb = g0; gb < g1; gb += 32) {
    const int g = gb + lane;
    float4 s = make_float4(0, 0, 0, 0);
    if (g < g1) {
#pragma unroll 8
      for (int k = k0; k < k1; ++k) add(s, __ldcg(p + (long long)k * 4096 + g));
    }
    tmp[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && g < g1) {
      for (int w = 1; w < 8; ++w) add(s, tmp[w][lane]);
      ((float4*)sum)[g] = s;
    }
    __syncthreads();
  }
}

__device__ __forceinline__ void cluster_meet() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the same shared address in block `rank` of the cluster, and a store to it
__device__ __forceinline__ uint32_t peer_of(uint32_t a, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void peer_store(uint32_t a, const uint4& v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// byte of columns 4 q .. of row r in a piece (swizzled: a warp writes by rows)
__device__ __forceinline__ uint32_t piece_at(int r, int q) { return r * 256 + ((q ^ r) << 4); }

// The blocks' shares of S meet in their cluster.  Every block's share stands in
// its planes of S, as pieces; each goes to the block that owns it, which adds it up
// over the blocks in order and stores it, as hi and lo, into every block's planes.
// Both ways a warp's stores are contiguous, or the network between the SMs takes
// them one by one.
__device__ __forceinline__ void thin_share(const OrthArgs& a, int c, int pieces, float f,
                                           const unsigned char* S, uint32_t ss) {
  const int own = (pieces + a.thin - 1) / a.thin;
  const unsigned char* in = S + 2 * IMG;
  __syncthreads();
  for (int it = threadIdx.x; it < pieces * (PIECE / 16); it += THIN_THREADS) {
    const int u = it / (PIECE / 16), to = u / own;
    peer_store(peer_of(ss + 2 * IMG + (c * own + u - to * own) * PIECE + it % (PIECE / 16) * 16, to),
               *(const uint4*)(S + it * 16));
  }
  cluster_meet();
  const int mine = min(own, pieces - c * own);
  for (int it = threadIdx.x; it < mine * 64; it += THIN_THREADS) {
    const int ul = it >> 6, r = it >> 3 & 7, q = it & 7;
    float v[8] = {};
#pragma unroll 4
    for (int k = 0; k < a.thin; ++k) {
      const unsigned char* p = in + (k * own + ul) * PIECE;
      const float4 x = *(const float4*)(p + piece_at(r, 2 * q));
      const float4 y = *(const float4*)(p + piece_at(r, 2 * q + 1));
      v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
      v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
    uint4 h, l;
    split2(v[0] * f, v[1] * f, h.x, l.x);
    split2(v[2] * f, v[3] * f, h.y, l.y);
    split2(v[4] * f, v[5] * f, h.z, l.z);
    split2(v[6] * f, v[7] * f, h.w, l.w);
    const int u = c * own + ul;
    const uint32_t at = ss + img_at((u & 15) * 8 + r, (u >> 4) * 64 + q * 8);
    for (int k = 0; k < a.thin; ++k) {
      const uint32_t to = peer_of(at, k);
      peer_store(to, h);
      peer_store(to + IMG, l);
    }
  }
  fence_proxy_async();  // (the tensor cores of every block read the planes)
  cluster_meet();
}

// How a matrix's blocks meet: there is one, or they are a cluster, or through
// global memory.
enum { ALONE, CLUSTER, GLOBAL };
template <int MEET>
__global__ void __launch_bounds__(THIN_THREADS, 1) k_orth_thin(const OrthArgs a) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ float4 tmp[8][32];
  __shared__ __align__(8) uint64_t bar[1];
  __shared__ uint32_t tmem_holder[1];
  __shared__ int abort_s;
  unsigned char* X = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char* S = X + 2 * IMG;  // S, then P
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = MEET == ALONE ? blockIdx.x : blockIdx.x / a.thin;
  const int c = MEET == ALONE ? 0 : blockIdx.x - b * a.thin;
  const int j0 = c * 128, nc = min(128, a.n - j0);
  // a warp's lanes are 32 rows; it takes every other 32 columns
  const int row = (warp & 3) * 32 + lane, cbase = (warp >> 2) * 32;
  if (tid == 0) {
    ptx::mbar_init(bar, 1);
    ptx::fence_mbar_init();
    abort_s = 0;
  }
  if (warp == 0) {
    ptx::tmem_alloc(tmem_holder, 256);
    ptx::tmem_relinquish();
  }
  if (a.in_f32) thin_load<float>(a, b, j0, X);
  else thin_load<__nv_bfloat16>(a, b, j0, X);
  ptx::tc_fence_before();
  __syncthreads();
  if (MEET == CLUSTER) cluster_meet();  // (the others run: their shared memory may be written)
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t xs = ptx::smem_u32(X), ss = ptx::smem_u32(S);
  const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const int mk = (a.m + 15) / 16, nk = (nc + 15) / 16;  // K steps over m and over the columns
  uint32_t parity = 0;
  // One product: thread 0 issues it once the block's writes are visible to the
  // tensor cores; afterwards the accumulator is there for every thread.
  auto product = [&](uint32_t pa, uint32_t pb, int b_mn, int n, int ksteps) {
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (tid == 0) {
      thin_mma(tmem, pa, pb, b_mn, n, ksteps);
      ptx::mma_commit(bar);
    }
    __syncwarp();
    if (!ptx::mbar_wait(bar, parity, a.wait_ns)) report(a.status, RNNT_ERR_TIMEOUT);
    __syncwarp();
    parity ^= 1;
    ptx::tc_fence_after();
  };
  auto acc32 = [&](int col0, float (&v)[32]) {
    float x[32];
    __syncwarp();  // (a warp reads tensor memory together: its rows past m stored nothing before)
    ptx::tmem_ld32(lanes + col0, v);
    ptx::tmem_ld32(lanes + 128 + col0, x);
    ptx::tmem_ld_wait();
    ptx::reg_fence32(v);
    ptx::reg_fence32(x);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += x[j];
  };
  unsigned arrivals = 0;
  auto meet = [&]() {
    __syncthreads();
    arrivals += a.thin;
    if (tid == 0) {
      if (!(a.lost && blockIdx.x == 0 && arrivals == a.thin))
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.counter + b) : "memory");
      if (!abort_s && !grid_wait(a, arrivals, &abort_s, b)) give_up(a, &abort_s);
    }
    __syncthreads();
  };
  float* part = a.part + (long long)b * a.thin * 128 * 128;
  float* sum = a.sum + (long long)b * 128 * 128;
#pragma unroll 1
  for (int step = 0; step < a.steps; ++step) {
    // S
    product(xs, xs, 0, mk * 16, nk);
    const float fs = 1.f / (1 << (2 * XE - SE));
    if constexpr (MEET == CLUSTER) {
#pragma unroll 1
      for (int c0 = cbase; c0 < mk * 16; c0 += 64) {
        float v[32];
        acc32(c0, v);
        // piece (64 columns) * 16 + (8 rows)
        unsigned char* p = S + ((c0 >> 6) * 16 + (row >> 3)) * PIECE;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *(float4*)(p + piece_at(row & 7, (c0 & 63) / 4 + i)) =
              make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
      thin_share(a, c, (mk * 16 + 63) / 64 * 16, fs, S, ss);
    } else if constexpr (MEET == GLOBAL) {  // (stored by columns: lanes are rows)
#pragma unroll 1
      for (int c0 = cbase; c0 < a.m; c0 += 64) {
        float v[32];
        acc32(c0, v);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c0 + j < a.m) part[((long long)c * 128 + c0 + j) * 128 + row] = v[j];
      }
      meet();
      thin_reduce(part, sum, c, a.thin, a.m, tmp);
      meet();
    }
#pragma unroll 1
    for (int c0 = cbase; c0 < mk * 16 && MEET != CLUSTER; c0 += 64) {
      float v[32];
      if constexpr (MEET == GLOBAL) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = c0 + j < a.m ? __ldcg(sum + (c0 + j) * 128 + row) : 0.f;
      } else {
        acc32(c0, v);
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = c0 + j < a.m ? v[j] * fs : 0.f;
      img_store(S, row, c0, v);
    }
    // P, over S
    product(ss, ss, 0, mk * 16, mk);
    const float ps = kB / (1 << (SE - PE)), pp = kC / (1 << (2 * SE - PE));
    const float d = shift_of(step) * (1 << PE);
#pragma unroll 1
    for (int c0 = cbase; c0 < mk * 16; c0 += 64) {
      float v[32], x[32];
      acc32(c0, v);
      img_load(S, row, c0, x);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        v[j] = fmaf(ps, x[j], v[j] * pp) - (row == c0 + j ? d : 0.f);
        if (row >= a.m || c0 + j >= a.m) v[j] = 0.f;
      }
      img_store(S, row, c0, v);
    }
    // X
    product(ss, xs, 1, nk * 16, mk);
    const float f = kA + shift_of(step);
#pragma unroll 1
    for (int c0 = cbase; c0 < nk * 16; c0 += 64) {
      float v[32], x[32];
      acc32(c0, v);
      img_load(X, row, c0, x);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        v[j] = fmaf(f, x[j], v[j] * (1.f / (1 << PE)));
        if (c0 + j >= nc) v[j] = 0.f;
      }
      if (step + 1 < a.steps) {
        img_store(X, row, c0, v);
        continue;
      }
      if (row < a.m) {
        const long long o = b * a.out_batch;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (c0 + j >= nc) continue;
          const long long at = o + (a.tall ? (j0 + c0 + j) * a.out_ld + row
                                           : row * a.out_ld + j0 + c0 + j);
          if (a.out_f32) ((float*)a.O)[at] = v[j] * (1.f / (1 << XE));
          else ((__nv_bfloat16*)a.O)[at] = __float2bfloat16_rn(v[j] * (1.f / (1 << XE)));
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 0) ptx::tmem_dealloc(tmem, 256);
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
  size_t w_X[2][2], w_S[2], w_P[2], w_part, w_sum, w_sums, w_sync, total;
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
  a.wait_ns = WAIT_NS;
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
  a.chunks = fast_div((uint32_t)cdiv(a.cols, 8));
  a.ldm = cdiv(a.m, 8) * 8;
  const long long nt = cdiv(a.m, BM);
  a.blocks = (int)(nt * (nt + 1) / 2);
  // exact products where the result is fp32; for small matrices they cost
  // little (a product's time is its latency); and past five steps, for which the
  // fast ones are made (see the head of this file)
  a.exact = a.out_f32 || a.m <= 256 || a.steps > 5;
  // gram: K in as many ranges as there are SMs for its blocks, eight K blocks
  // at least (a range's partial tile costs as much as four); without ranges,
  // and for poly, 64-wide tiles while they fit the SMs once: a product's time
  // is then a tile's, and half the tile takes half of it
  const int kbs = (int)cdiv(a.n, BK);
  const long long gu = (long long)a.batch * a.blocks;
  a.splits = (int)std::max<long long>(1, std::min<long long>(kSms / std::max(1LL, gu), kbs / 8));
  a.kb_split = (int)cdiv(kbs, a.splits);
  a.splits = (int)cdiv(kbs, a.kb_split);
  a.bn[POLY] = 2 * gu <= kSms ? 64 : 128;
  a.bn[GRAM] = a.splits == 1 ? a.bn[POLY] : 128;
  // update: the width whose rounds over the SMs load the fewest operand rows (an
  // SM takes in about 96 GB/s whatever the stage, which bounds every product
  // here); exact ones keep a second accumulator: 128 at most
  const int un = a.tall ? a.m : a.n, um = a.tall ? a.n : a.m;
  a.ut_m = (int)cdiv(um, BM);
  auto tiles = [&](int bn) { return (long long)a.batch * a.ut_m * cdiv(un, bn); };
  // the tiles of the last round go out as two halves each where the SMs take them
  // at once (16384 x 1024, 512 tiles of 256: 420 us, in whole rounds 440)
  auto halved = [&](int bn) {
    const long long rest = tiles(bn) % kSms;
    return tiles(bn) > kSms && bn >= 128 && 2 * rest <= kSms &&
                   (un - 1) % bn >= bn / 2 ? rest : 0;
  };
  auto rows = [&](int bn) {
    return cdiv(tiles(bn), kSms) * (BM + bn) - (halved(bn) ? bn / 2 : 0);
  };
  a.bn[UPDATE] = 64;
  for (int bn = 128; bn <= (a.exact ? 128 : 256); bn *= 2)
    if (rows(bn) < rows(a.bn[UPDATE])) a.bn[UPDATE] = bn;
  a.ut_n = (int)cdiv(un, a.bn[UPDATE]);
  a.ut_whole = (int)(tiles(a.bn[UPDATE]) - halved(a.bn[UPDATE]));
  const long long gram_units = gu * (BM / a.bn[GRAM]) * a.splits;
  const long long units = std::max(
      {gram_units, gu * (BM / a.bn[POLY]), (long long)a.batch * a.ut_m * a.ut_n});
  if (tiles(64) > 2147483647LL || gram_units * 64 > 2147483647LL) return false;
  p->ctas = (int)std::min<long long>(kSms, units);
  // (two blocks an SM at most: every warp that scales X adds up these sums; 1216
  // of them, 412 us for 16384 x 1024, were slower than 304, 405)
  a.nb = (int)std::min<long long>(std::max<long long>(1, (long long)a.rows * a.cols / 8192),
                                  2 * kSms);
  // thin: a block per 128 columns; more than one per matrix wait for one another
  // and have to be resident together
  const long long thin = cdiv(a.n, 128);
  a.thin = a.m <= 128 && (thin == 1 || thin * a.batch <= kSms) ? (int)thin : 0;
  const size_t x = a.thin ? 0 : 2 * (size_t)a.batch * a.rows * a.ldx;
  const size_t s = a.thin ? 0 : 2 * (size_t)a.batch * a.m * a.ldm;
  size_t o = 0;
  auto put = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes); return at; };
  // (fast products read no lo of X: its only reader is the thread that writes the
  // new one, so one plane serves both buffers, and X of 16384 x 1024 stays in L2)
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      p->w_X[i][j] = i && j && !a.exact ? p->w_X[0][1] : put(x);
  for (int j = 0; j < 2; ++j) p->w_S[j] = put(s);
  for (int j = 0; j < 2; ++j) p->w_P[j] = put(s);
  p->w_part = put(a.thin > 1 ? 4 * (size_t)a.batch * a.thin * 128 * 128
                  : !a.thin && a.splits > 1 ? 4 * (size_t)gram_units * BM * a.bn[GRAM] : 0);
  p->w_sum = put(a.thin > 1 ? 4 * (size_t)a.batch * 128 * 128 : 0);
  p->w_sums = put(8 * (size_t)a.batch * a.nb);
  p->w_sync = put(4 * (size_t)a.batch + 4);
  p->total = o;
  return true;
}

// Blocks that wait for one another are all resident at once: a cooperative launch.
template <int WHICH, typename... KA, typename... A>
cudaError_t launch_resident(void (*k)(KA...), bool together, int grid, int threads, size_t smem,
                            cudaStream_t st, const A&... args) {
  static std::atomic<bool> opted_in[kDeviceSlots];  // per kernel (WHICH) and device
  std::atomic<bool>& opted = opted_in[device_slot()];
  if (!opted.load()) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    opted.store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = together ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// The blocks of a thin matrix as a cluster, where the card can hold one (*done).
cudaError_t launch_thin_cluster(const OrthArgs& a, cudaStream_t st, bool* done) {
  static std::atomic<int> fits[kDeviceSlots][MAX_THIN_CLUSTER + 1];  // 0: not asked, 1: no, 2: yes
  *done = false;
  if (a.thin < 2 || a.thin > MAX_THIN_CLUSTER) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = a.thin;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(a.thin * a.batch);
  cfg.blockDim = dim3(THIN_THREADS);
  cfg.dynamicSmemBytes = THIN_CLUSTER_SMEM;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  std::atomic<int>& f = fits[device_slot()][a.thin];
  if (!f.load()) {
    auto k = k_orth_thin<CLUSTER>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         THIN_CLUSTER_SMEM);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k_orth_thin<CLUSTER>, &cfg) != cudaSuccess) {
      cudaGetLastError();  // (no cluster of this size: not an error of the call)
      n = 0;
    }
    f.store(n > 0 ? 2 : 1);
  }
  if (f.load() != 2) return cudaSuccess;
  *done = true;
  return cudaLaunchKernelEx(&cfg, k_orth_thin<CLUSTER>, a);
}

cudaError_t orth_launch(OrthPlan& p, cudaStream_t st) {
  OrthArgs& a = p.a;
  double* sums = const_cast<double*>(a.sums);
  const dim3 grid(a.nb, a.batch);
  if (a.in_f32) k_orth_sumsq<float><<<grid, 256, 0, st>>>(a, sums);
  else k_orth_sumsq<__nv_bfloat16><<<grid, 256, 0, st>>>(a, sums);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  bool done = false;
  if ((e = launch_thin_cluster(a, st, &done)) != cudaSuccess || done) return e;
  if (a.thin)
    return a.thin > 1
               ? launch_resident<3>(k_orth_thin<GLOBAL>, true, a.thin * a.batch, THIN_THREADS,
                                    THIN_SMEM, st, a)
               : launch_resident<2>(k_orth_thin<ALONE>, false, a.batch, THIN_THREADS, THIN_SMEM,
                                    st, a);
  OrthMaps maps;
  for (int j = 0; j < 2; ++j) {
    for (int i = 0; i < 2; ++i)
      if (!make_map(&maps.m[i][j], a.X[i][j], a.rows, a.cols, a.ldx, a.batch))
        return cudaErrorInvalidValue;
    if (!make_map(&maps.m[BUF_S][j], a.S[j], a.m, a.m, a.ldm, a.batch) ||
        !make_map(&maps.m[BUF_P][j], a.P[j], a.m, a.m, a.ldm, a.batch))
      return cudaErrorInvalidValue;
  }
  const int blocks = std::min(p.ctas, num_sms());
  return a.exact ? launch_resident<1>(k_orth<1>, true, blocks, THREADS, SMEM, st, maps, a)
                 : launch_resident<0>(k_orth<0>, true, blocks, THREADS, SMEM, st, maps, a);
}

rnnt_status orth_call(const rnnt_orth_dims* dims, OrthPlan& p, const void* G, void* O, void* ws,
                      size_t ws_bytes, int32_t* status, rnnt_stream stream) {
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
  a.sum = (float*)(w + p.w_sum);
  a.sums = (const double*)(w + p.w_sums);
  a.counter = (unsigned*)(w + p.w_sync);
  a.abort = (int*)(w + p.w_sync) + a.batch;
  a.G = G; a.O = O; a.status = status;
  const int per16 = a.out_f32 ? 4 : 8;
  a.out_vec = aligned_to(O, 16) && a.cols % per16 == 0 && a.out_ld % per16 == 0 &&
              (a.batch == 1 || a.out_batch % per16 == 0);
  cudaStream_t st = (cudaStream_t)stream;
  ProfScope ps("orth", st);
  ps.set_kernels(2);
  OPS_CHECK(orth_launch(p, st));
  return RNNT_OK;
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
  return orth_call(dims, p, G, O, ws, ws_bytes, status, stream);
}

rnnt_status rnnt_testing_orth_timeout(const rnnt_orth_dims* dims, const void* G, void* O, void* ws,
                                      size_t ws_bytes, int32_t* status,
                                      unsigned long long wait_ns, rnnt_stream stream) {
  OrthPlan p;
  // (the blocks of a cluster, or one alone, meet at no barrier that gives up)
  if (!orth_plan(dims, &p) || p.a.thin == 1 || (p.a.thin && p.a.thin <= MAX_THIN_CLUSTER))
    return RNNT_ERR_INVALID_ARG;
  p.a.wait_ns = wait_ns;
  p.a.lost = 1;
  return orth_call(dims, p, G, O, ws, ws_bytes, status, stream);
}

rnnt_status rnnt_testing_orth_plan(const rnnt_orth_dims* dims, rnnt_testing_orth* out) {
  OrthPlan p;
  if (!out || !orth_plan(dims, &p)) return RNNT_ERR_INVALID_ARG;
  const OrthArgs& a = p.a;
  *out = {};
  out->thin = a.thin;
  out->exact = a.exact;
  out->splits = a.splits;
  const int sym = a.batch * a.blocks, tiles = a.batch * a.ut_m * a.ut_n;
  for (int k = 0; k < 3; ++k) out->bn[k] = a.bn[k];
  out->units[GRAM] = sym * (BM / a.bn[GRAM]) * a.splits;
  out->units[POLY] = sym * (BM / a.bn[POLY]);
  out->units[UPDATE] = 2 * tiles - a.ut_whole;
  out->halved = tiles - a.ut_whole;
  out->blocks = a.thin ? a.thin * a.batch : p.ctas;
  return RNNT_OK;
}

}  // extern "C"
