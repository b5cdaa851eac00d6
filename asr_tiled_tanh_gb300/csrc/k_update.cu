// k_update.cu -- gradient clipping and the AdamW update over lists of tensors
// (include/rnnt_ops.h).
#include <algorithm>
#include <atomic>
#include <climits>
#include <memory>
#include <new>
#include <type_traits>

#include "../../include/rnnt_testing.h"
#include "ops.h"
#include "ptx.cuh"

namespace rnnt {
namespace {

constexpr int UT = 256;       // threads
constexpr int CHUNK = 8192;   // elements of one tensor that a block takes at a time
constexpr int PARTS = 1024;   // sums of squares that the workspace holds
// Tensors a launch: its tables are kernel parameters, of which there are 32 KB.  (The
// host's part of a call on 296 tensors: 14 us with one table of 512, 17 with two
// launches of 256 and 64.)
constexpr int FEW = 32, MANY = 512;

// A launch's tensors, cut into chunks that are numbered through.
template <int N>
struct Chunks {
  int n;
  int first[N + 1];  // chunks before each tensor
  long long count[N];
  uint8_t bf16[N];   // the gradient's type
  // elements before the first four that lie on 16 bytes (8 of bf16): of the gradient, for
  // AdamW of all the tensors of the place (views of buffers that are laid out alike), -1
  // where they differ
  int8_t head[N];
};

// Chunks first, first + step, ... (step < 0: downwards) and the one at hand.
template <int N>
struct Walk {
  int k, step, i;  // the chunk, its tensor
  long long at;    // its first element, and their number
  int n;
  __device__ __forceinline__ Walk(const Chunks<N>& c, int first, int step_)
      : k(first), step(step_), i(step_ < 0 ? c.n - 1 : 0) {
    if (on(c)) find(c);
  }
  __device__ __forceinline__ bool on(const Chunks<N>& c) const {
    return k >= 0 && k < c.first[c.n];
  }
  __device__ __forceinline__ void find(const Chunks<N>& c) {
    while (k >= c.first[i + 1]) ++i;
    while (k < c.first[i]) --i;
    at = (long long)(k - c.first[i]) * CHUNK;
    n = (int)min((long long)CHUNK, c.count[i] - at);
  }
  __device__ __forceinline__ void next(const Chunks<N>& c) {
    k += step;
    if (on(c)) find(c);
  }
};
// The block's, from the last on: an earlier pass left those in L2.
template <int N>
__device__ __forceinline__ Walk<N> backwards(const Chunks<N>& c) {
  return Walk<N>(c, c.first[c.n] - 1 - (int)blockIdx.x, -(int)gridDim.x);
}

// Four elements of a gradient as they are stored.
template <bool BF16>
struct Quad {
  using U = std::conditional_t<BF16, uint2, float4>;
  static __device__ __forceinline__ U load(const void* g, long long i) {
    return BF16 ? *(const U*)((const __nv_bfloat16*)g + i) : *(const U*)((const float*)g + i);
  }
  static __device__ __forceinline__ float4 widen(const U& u) {
    if constexpr (BF16)
      return make_float4(ptx::bf16lo(u.x), ptx::bf16hi(u.x), ptx::bf16lo(u.y), ptx::bf16hi(u.y));
    else
      return u;
  }
};
__device__ __forceinline__ uint2 pack4(const float4& q) {
  return make_uint2(ptx::pack_bf16x2(q.x, q.y), ptx::pack_bf16x2(q.z, q.w));
}
// One element.
template <bool BF16>
__device__ __forceinline__ float grad1(const void* g, long long i) {
  return BF16 ? __bfloat162float(((const __nv_bfloat16*)g)[i]) : ((const float*)g)[i];
}

// Sum of v over the block's threads in a fixed order, for the first warp's.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v, double* scr) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) scr[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < THREADS / 32 ? scr[threadIdx.x] : 0.;
#pragma unroll
    for (int d = THREADS / 64; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  }
  return v;
}

// ---- norm -------------------------------------------------------------------------
// A thread's 32 elements of a chunk: squares added in fp32 (two chains of 16 terms of one
// sign, and their sum), in fp64 where that left the range or came near its bottom.  fp64 for
// every element would cost three times what DRAM does.
constexpr int EACH = CHUNK / UT;
__device__ __forceinline__ double squares(const float (&g)[EACH]) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < EACH; k += 2) {
    const float2 v = make_float2(g[k], g[k + 1]);
    s = __ffma2_rn(v, v, s);
  }
  const float t = s.x + s.y;
  if (t >= 0x1p-60f && t <= 0x1p126f) return t;
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < EACH; ++k) any |= __float_as_uint(g[k]) << 1;
  if (!any) return 0;
  // (unrolled whole: a loop would have every thread's elements in local memory, 55 us for
  // 25 of 68M in bf16)
  double d = 0;
#pragma unroll
  for (int k = 0; k < EACH; ++k) d = fma((double)g[k], (double)g[k], d);
  return d;
}

// A chunk's n elements, by fours from `head` on (head < 0: none) and the others, at most
// six: other(i) for i below `others`.
struct Cut {
  int head, whole, others;
  __device__ __forceinline__ Cut(int n, int h) {
    head = min(max(h, 0), n);
    whole = h < 0 ? 0 : (n - head) & ~3;
    others = n - whole;
  }
  __device__ __forceinline__ int other(int i) const { return i < head ? i : whole + i; }
};

// The squares of a chunk's n elements from `at` on: a thread's loads all under way
// before the first is used.  (A gradient alone always has a head.)
template <bool BF16>
__device__ __forceinline__ double chunk_squares(const void* g, long long at, int n, int head,
                                                int tid) {
  using Q = Quad<BF16>;
  float v[EACH];
  const Cut c(n, head);
  typename Q::U u[EACH / 4];
#pragma unroll
  for (int j = 0; j < EACH / 4; ++j) {
    const int e = (j * UT + tid) * 4;
    u[j] = typename Q::U{};
    if (e < c.whole) u[j] = Q::load(g, at + c.head + e);
  }
#pragma unroll
  for (int j = 0; j < EACH / 4; ++j) {
    const float4 q = Q::widen(u[j]);
    v[4 * j] = q.x;
    v[4 * j + 1] = q.y;
    v[4 * j + 2] = q.z;
    v[4 * j + 3] = q.w;
  }
  double d = squares(v);
  if (tid < c.others) {
    const double q = grad1<BF16>(g, at + c.other(tid));
    d += q * q;
  }
  return d;
}

__device__ __forceinline__ float2 norm_and_scale(double sum, float max_norm, float eps) {
  // (a root and a quotient in fp64 cost 0.7 us where a thread waits for them alone)
  if (sum >= 0x1p-100 && sum <= 0x1p100) {
    const float norm = sqrtf((float)sum), q = max_norm / (norm + eps);
    return make_float2(norm, q >= 1.f ? 1.f : q);
  }
  // (a norm that fp32 does not hold is infinite, and the scale goes with it)
  const double norm = sqrt(sum), q = (double)max_norm / (norm + (double)eps);
  if (isinf((float)norm)) return make_float2(INFINITY, 0.f);
  return make_float2((float)norm, q >= 1 ? 1.f : (float)q);  // (NaN stays)
}

template <int N>
struct NormTable {
  Chunks<N> c;
  const void* g[N];
};

// part[block]: the block's sum of squares (added to what an earlier launch of the
// same call left there).
template <int N>
__global__ void __launch_bounds__(UT)
k_clip_squares(const __grid_constant__ NormTable<N> t, double* __restrict__ part, int add) {
  __shared__ double scr[UT / 32];
  ptx::griddep_launch();
  double sum = 0;
#pragma unroll 1
  for (Walk<N> w(t.c, blockIdx.x, gridDim.x); w.on(t.c); w.next(t.c)) {
    const void* g = t.g[w.i];
    const int head = t.c.head[w.i];
    sum += t.c.bf16[w.i] ? chunk_squares<true>(g, w.at, w.n, head, threadIdx.x)
                         : chunk_squares<false>(g, w.at, w.n, head, threadIdx.x);
  }
  sum = block_sum<UT>(sum, scr);
  if (threadIdx.x == 0) part[blockIdx.x] = add ? part[blockIdx.x] + sum : sum;
}

// What the sums of squares and the limit make of it, for the block's first thread.
struct NormArgs {
  const double* part;
  int n;  // sums; 0: an earlier launch has left (norm, scale) in clip
  float max_norm, eps;
  float* clip;
};
__device__ __forceinline__ float2 clip_of(const NormArgs& a, double* scr) {
  double sum = 0;
#pragma unroll
  for (int k = 0; k < PARTS / UT; ++k)
    if (threadIdx.x + k * UT < a.n) sum += __ldcg(a.part + threadIdx.x + k * UT);
  sum = block_sum<UT>(sum, scr);
  float2 c = make_float2(0.f, 0.f);
  if (threadIdx.x == 0) c = norm_and_scale(sum, a.max_norm, a.eps);
  return c;
}

__global__ void __launch_bounds__(UT)
k_clip_norm(NormArgs a) {
  __shared__ double scr[UT / 32];
  ptx::griddep_launch();
  ptx::griddep_wait();
  const float2 c = clip_of(a, scr);
  if (threadIdx.x == 0) {
    a.clip[0] = c.x;
    a.clip[1] = c.y;
  }
}

// ---- scaling ----------------------------------------------------------------------
template <int N>
struct ScaleTable {
  Chunks<N> c;  // (heads of the gradients alone: the squares are added in their order)
  const void* g[N];
  void* into[N];
  uint8_t alike[N];  // the other tensor lies as the gradient does
  __device__ __forceinline__ int head(int i) const { return alike[i] ? c.head[i] : -1; }
};

// Single elements under way, where the places differ (68M in bf16 with the norm, 281 us
// one by one, 189 two together, 141 four, 145 eight, which spill).
constexpr int SINGLES = 4;
template <bool BF16>
__device__ __forceinline__ void scale_chunk(const void* g, void* into, long long at, int n,
                                            int head, float s, int tid) {
  using Q = Quad<BF16>;
  const Cut c(n, head);
  if (c.whole) {
    typename Q::U u[EACH / 4];
#pragma unroll
    for (int j = 0; j < EACH / 4; ++j) {
      const int e = (j * UT + tid) * 4;
      if (e < c.whole) u[j] = Q::load(g, at + c.head + e);
    }
#pragma unroll
    for (int j = 0; j < EACH / 4; ++j) {
      const int e = (j * UT + tid) * 4;
      if (e >= c.whole) continue;
      const long long to = at + c.head + e;
      float4 q = Q::widen(u[j]);
      q = make_float4(s * q.x, s * q.y, s * q.z, s * q.w);
      if constexpr (BF16) *(uint2*)((__nv_bfloat16*)into + to) = pack4(q);
      else *(float4*)((float*)into + to) = q;
    }
  }
#pragma unroll 1
  for (int i0 = tid; i0 < c.others; i0 += SINGLES * UT) {
    float v[SINGLES];
#pragma unroll
    for (int j = 0; j < SINGLES; ++j)
      if (i0 + j * UT < c.others) v[j] = s * grad1<BF16>(g, at + c.other(i0 + j * UT));
#pragma unroll
    for (int j = 0; j < SINGLES; ++j) {
      if (i0 + j * UT >= c.others) continue;
      const long long e = at + c.other(i0 + j * UT);
      if constexpr (BF16) ((__nv_bfloat16*)into)[e] = __float2bfloat16_rn(v[j]);
      else ((float*)into)[e] = v[j];
    }
  }
}

// Every block adds up the sums of squares for itself: 8 KB from L2, where another launch
// between them takes 2 us.  (Three blocks an SM: 336M elements in bf16 312 us with the
// norm, 340 with two, 314 with four, 323 with five; 4.7M in fp32 14.0, 13.4, 15.1, 17.6.)
template <int N>
__global__ void __launch_bounds__(UT, 3)
k_clip_scale(const __grid_constant__ ScaleTable<N> t, NormArgs a) {
  __shared__ double scr[UT / 32];
  __shared__ float scale_s;
  ptx::griddep_wait();
  if (a.n) {
    const float2 c = clip_of(a, scr);
    if (threadIdx.x == 0) {
      scale_s = c.y;
      if (blockIdx.x == 0) {
        a.clip[0] = c.x;
        a.clip[1] = c.y;
      }
    }
    __syncthreads();
  }
  const float s = a.n ? scale_s : __ldcg(a.clip + 1);
#pragma unroll 1
  for (Walk<N> w = backwards(t.c); w.on(t.c); w.next(t.c)) {
    const void* g = t.g[w.i];
    void* into = t.into[w.i];
    const int head = t.head(w.i);
    if (s == 1.f && g == into) continue;
    if (t.c.bf16[w.i]) scale_chunk<true>(g, into, w.at, w.n, head, s, threadIdx.x);
    else scale_chunk<false>(g, into, w.at, w.n, head, s, threadIdx.x);
  }
}

// ---- short lists --------------------------------------------------------------------
// Norm and scaling in one launch of one cluster: its blocks add up each other's sums
// in shared memory.  A program that calls for few elements waits for its host, which a
// launch costs 2.4 us (eight tensors of 14 thousand elements 12.2 us as called from
// Python, 16.0 in two launches; on the GPU alone 6.9 and 5.6, 200 thousand 7.2 and 5.2).
constexpr int CBLOCKS = 16, CGROUPS = 2;  // blocks at most, and their groups of UT threads
// What one cluster takes in one launch: up to as many chunks (262,144 elements) as its
// groups of threads take once.
constexpr int SHORT = CBLOCKS * CGROUPS;

// value at the same shared address of another block of the cluster
__device__ __forceinline__ double peer_f64(const double* mine, int rank) {
  uint32_t at;
  double v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at) : "r"(ptx::smem_u32(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// (into[0] NULL: the norm alone)
__global__ void __launch_bounds__(UT * CGROUPS)
k_clip_short(const __grid_constant__ ScaleTable<SHORT> t, float max_norm, float eps,
             float* __restrict__ clip) {
  __shared__ double scr[UT * CGROUPS / 32], mine;
  __shared__ float scale_s;
  ptx::griddep_launch();
  const int tid = threadIdx.x & (UT - 1), group = threadIdx.x / UT;
  const int first = blockIdx.x * CGROUPS + group, step = gridDim.x * CGROUPS;
  double sum = 0;
#pragma unroll 1
  for (Walk<SHORT> w(t.c, first, step); w.on(t.c); w.next(t.c)) {
    const void* g = t.g[w.i];
    const int head = t.c.head[w.i];
    sum += t.c.bf16[w.i] ? chunk_squares<true>(g, w.at, w.n, head, tid)
                         : chunk_squares<false>(g, w.at, w.n, head, tid);
  }
  sum = block_sum<UT * CGROUPS>(sum, scr);
  if (threadIdx.x == 0) mine = sum;
  cluster_sync();
  if (threadIdx.x < 32) {
    sum = threadIdx.x < gridDim.x ? peer_f64(&mine, threadIdx.x) : 0.;
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (threadIdx.x == 0) {
      const float2 c = norm_and_scale(sum, max_norm, eps);
      scale_s = c.y;
      if (blockIdx.x == 0) {
        clip[0] = c.x;
        clip[1] = c.y;
      }
    }
  }
  cluster_sync();  // (and no block leaves while its sum is read)
  if (!t.into[0]) return;
  const float s = scale_s;
#pragma unroll 1
  for (Walk<SHORT> w(t.c, first, step); w.on(t.c); w.next(t.c)) {
    const void* g = t.g[w.i];
    void* into = t.into[w.i];
    const int head = t.head(w.i);
    if (s == 1.f && g == into) continue;
    if (t.c.bf16[w.i]) scale_chunk<true>(g, into, w.at, w.n, head, s, tid);
    else scale_chunk<false>(g, into, w.at, w.n, head, s, tid);
  }
}

// ---- AdamW ------------------------------------------------------------------------
template <int N>
struct AdamTable {
  Chunks<N> c;
  const void* g[N];
  float *p[N], *m[N], *v[N];
  __nv_bfloat16* low[N];
  float decay[N];
};

struct AdamArgs {
  float b1, b2, nb1, nb2;  // betas and 1 - beta
  float log1, log2;        // their logarithms
  float eps, lr;
  const float* lr_dev;
  const float* clip;
  int32_t* steps;
  int last;  // the call's last launch counts the update
};

struct AdamStep {
  float b1, b2, nb1, nb2, scale, eps, lr, r1, r2, decay;
  __device__ __forceinline__ void operator()(float& p, float& m, float& v, float g) const {
    g *= scale;
    m = fmaf(b1, m, nb1 * g);
    v = fmaf(b2, v, nb2 * g * g);
    p -= lr * fmaf(decay, p, (m * r1) / (sqrtf(v * r2) + eps));
  }
  __device__ __forceinline__ void operator()(float4& p, float4& m, float4& v,
                                             const float4& g) const {
    (*this)(p.x, m.x, v.x, g.x);
    (*this)(p.y, m.y, v.y, g.y);
    (*this)(p.z, m.z, v.z, g.z);
    (*this)(p.w, m.w, v.w, g.w);
  }
};

// Quads of each tensor that a thread has under way (336M elements: 1,764 us with the
// norm for one, 1,715 for two, 1,895 for four, which leave one block an SM less).
constexpr int AHEAD = 2;
// (and single elements, where the tensors' places differ: 68M, 712 us one by one, 511 two
// together, 561 three, 574 four)
constexpr int ONES = 2;

// A chunk's parts of p, m, v and low (or NULL).
struct Tensors {
  float *p, *m, *v;
  __nv_bfloat16* low;
};
template <bool BF16>
__device__ __forceinline__ void adam_chunk(const Tensors& x, const void* g, long long at, int n,
                                           int head, const AdamStep& f) {
  using Q = Quad<BF16>;
  const Cut c(n, head);
#pragma unroll 1
  for (int e0 = threadIdx.x * 4; e0 < c.whole; e0 += AHEAD * UT * 4) {
    float4 p[AHEAD], m[AHEAD], v[AHEAD];
    typename Q::U u[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int e = c.head + e0 + j * UT * 4;
      if (e0 + j * UT * 4 >= c.whole) continue;
      p[j] = *(const float4*)(x.p + e);
      m[j] = *(const float4*)(x.m + e);
      v[j] = *(const float4*)(x.v + e);
      u[j] = Q::load(g, at + e);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int e = c.head + e0 + j * UT * 4;
      if (e0 + j * UT * 4 >= c.whole) continue;
      f(p[j], m[j], v[j], Q::widen(u[j]));
      *(float4*)(x.p + e) = p[j];
      *(float4*)(x.m + e) = m[j];
      *(float4*)(x.v + e) = v[j];
      if (x.low) *(uint2*)(x.low + e) = pack4(p[j]);
    }
  }
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < c.others; i0 += ONES * UT) {
    float p[ONES], m[ONES], v[ONES], u[ONES];
#pragma unroll
    for (int j = 0; j < ONES; ++j) {
      const int e = c.other(i0 + j * UT);
      if (i0 + j * UT >= c.others) continue;
      p[j] = x.p[e];
      m[j] = x.m[e];
      v[j] = x.v[e];
      u[j] = grad1<BF16>(g, at + e);
    }
#pragma unroll
    for (int j = 0; j < ONES; ++j) {
      const int e = c.other(i0 + j * UT);
      if (i0 + j * UT >= c.others) continue;
      f(p[j], m[j], v[j], u[j]);
      x.p[e] = p[j];
      x.m[e] = m[j];
      x.v[e] = v[j];
      if (x.low) x.low[e] = __float2bfloat16_rn(p[j]);
    }
  }
}

// Bound by DRAM: 28 to 30 bytes an element in 8 streams.  (Two blocks an SM, so that the
// loads stay together: 336M elements 1,719 us with the norm, 1,743 where the compiler is
// left to it, 1,729 with three.)
template <int N>
__global__ void __launch_bounds__(UT, 2)
k_adamw(const __grid_constant__ AdamTable<N> t, AdamArgs a) {
  ptx::griddep_wait();
  // (a count at its end stays there)
  const int now = min(__ldcg(a.steps), INT_MAX - 1) + 1;
  const bool take = !a.clip || isfinite(__ldcg(a.clip));
  if (take) {
    AdamStep f;
    f.b1 = a.b1; f.b2 = a.b2; f.nb1 = a.nb1; f.nb2 = a.nb2; f.eps = a.eps;
    f.scale = a.clip ? __ldcg(a.clip + 1) : 1.f;
    f.lr = a.lr_dev ? __ldcg(a.lr_dev) : a.lr;
    // 1 - beta^t without the cancellation
    f.r1 = 1.f / -expm1f((float)now * a.log1);
    f.r2 = 1.f / -expm1f((float)now * a.log2);
#pragma unroll 1
    for (Walk<N> w = backwards(t.c); w.on(t.c); w.next(t.c)) {
      const Tensors x{t.p[w.i] + w.at, t.m[w.i] + w.at, t.v[w.i] + w.at,
                      t.low[w.i] ? t.low[w.i] + w.at : nullptr};
      f.decay = t.decay[w.i];
      if (t.c.bf16[w.i]) adam_chunk<true>(x, t.g[w.i], w.at, w.n, t.c.head[w.i], f);
      else adam_chunk<false>(x, t.g[w.i], w.at, w.n, t.c.head[w.i], f);
    }
  }
  // The last block to come here counts the update, when every block has read the
  // count, and the second word wraps to 0.
  __syncthreads();
  if (threadIdx.x) return;
  __threadfence();
  if (atomicInc((unsigned*)a.steps + 1, gridDim.x - 1) == gridDim.x - 1 && a.last && take)
    a.steps[0] = now;
}

// ---- host ----------------------------------------------------------------------
constexpr int MAX_TENSORS = 1 << 16;

bool list_ok(const rnnt_grad_list* l) {
  if (!l || l->n < 0 || l->n > MAX_TENSORS || (l->n && !l->count)) return false;
  for (int i = 0; i < l->n; ++i) {
    // (chunk numbers and byte offsets of a call stay within their types)
    if (l->count[i] < 0 || l->count[i] > (1LL << 36)) return false;
    if (l->dtype && !op_dtype(l->dtype[i])) return false;
  }
  return true;
}

bool is_bf16(const rnnt_grad_list* l, int i) { return l->dtype && l->dtype[i] == RNNT_BF16; }

// A tensor list's pointers: present and aligned where there are elements.
bool pointers_ok(const rnnt_grad_list* l, const void* const* p, bool grads) {
  if (!p) return l->n == 0;
  for (int i = 0; i < l->n; ++i)
    if (l->count[i] && (!p[i] || !aligned_to(p[i], grads && is_bf16(l, i) ? 2 : 4))) return false;
  return true;
}

// Memory that a call writes, and what must stay clear of it.  Lists whose tensors lie
// one after another in memory, as views of one buffer do, are runs that need no sorting
// (1,480 pieces: 25 us to sort, which is what the GPU takes for a small model).
struct Span {
  uintptr_t from, to;
  bool written;
};
class Spans {
 public:
  // (the thread keeps the memory)
  explicit Spans(size_t most) {
    static thread_local std::unique_ptr<Span[]> kept;
    static thread_local size_t room = 0;
    if (!kept || most > room) {
      kept.reset(new (std::nothrow) Span[most + 64]);
      room = kept ? most + 64 : 0;
    }
    s_ = kept.get();
  }
  bool ok() const { return s_ != nullptr; }
  // n pieces: at(i), bytes(i) each, or none of them
  template <typename P, typename B>
  void add(int n, bool written, P at, B bytes) {
    Span* to = s_ + n_;
    uintptr_t last = ~(uintptr_t)0;  // (a list begins a run)
    for (int i = 0; i < n; ++i) {
      const uintptr_t from = (uintptr_t)at(i);
      const size_t size = bytes(i);
      if (!from || !size) continue;
      if (from < last && ++runs_ <= RUNS) run_[runs_ - 1] = to - s_;
      last = from;
      *to++ = {from, from + size, written};
    }
    n_ = to - s_;
  }
  // whether a written one meets another
  bool overlap() {
    bool sorted = runs_ <= RUNS;
    int order[RUNS];
    if (sorted) {
      run_[runs_] = n_;
      for (int k = 0; k < runs_; ++k) order[k] = k;
      std::sort(order, order + runs_,
                [&](int a, int b) { return s_[run_[a]].from < s_[run_[b]].from; });
      for (int k = 1; k < runs_; ++k)
        sorted &= s_[run_[order[k - 1] + 1] - 1].from <= s_[run_[order[k]]].from;
    }
    uintptr_t reach[2] = {0, 0};  // of what was read, of what was written
    if (!sorted) {
      std::sort(s_, s_ + n_, [](const Span& a, const Span& b) { return a.from < b.from; });
      return meets(s_, s_ + n_, reach);
    }
    for (int k = 0; k < runs_; ++k)
      if (meets(s_ + run_[order[k]], s_ + run_[order[k] + 1], reach)) return true;
    return false;
  }

 private:
  static constexpr int RUNS = 8;
  Span* s_;
  size_t n_ = 0, run_[RUNS + 1];  // where runs of ascending places begin
  int runs_ = 0;
  static bool meets(const Span* a, const Span* end, uintptr_t (&reach)[2]) {
    uintptr_t read = reach[0], written = reach[1];
    for (; a < end; ++a) {
      if (a->from < written || (a->written && a->from < read)) return true;
      if (a->written) written = std::max(written, a->to);
      else read = std::max(read, a->to);
    }
    reach[0] = read;
    reach[1] = written;
    return false;
  }
};

// Elements before the first four that lie together in p (0 to 3).
int head_of(const void* p, bool bf16) {
  return (int)((4 - (uintptr_t)p / (bf16 ? 2 : 4) % 4) % 4);
}

// The next launch's tensors, from i on, into c; fill(k, j): tensor j is its k-th, and
// returns its head.  Returns the tensor after them.
template <int N, typename F>
int next_chunks(const rnnt_grad_list* l, int i, Chunks<N>* c, F fill) {
  c->n = 0;
  c->first[0] = 0;
  for (; i < l->n && c->n < N; ++i) {
    if (!l->count[i]) continue;
    const long long chunks = cdiv(l->count[i], CHUNK);
    if (c->n && c->first[c->n] + chunks > (1 << 30)) break;
    const int k = c->n++;
    c->count[k] = l->count[i];
    c->bf16[k] = is_bf16(l, i);
    c->first[k + 1] = c->first[k] + (int)chunks;
    c->head[k] = (int8_t)fill(k, i);
  }
  return i;
}

// Blocks of a kernel that the card holds at a time, asked once per kernel and device.
template <typename K>
cudaError_t resident(K k, std::atomic<int>* known, int* out) {
  std::atomic<int>& m = known[device_slot()];
  *out = m.load();
  if (*out) return cudaSuccess;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, k, UT, 0);
  if (e != cudaSuccess) return e;
  *out = std::max(1, *out) * num_sms();
  m.store(*out);
  return e;
}

// A launch; dep: its blocks come in under the tail of the kernel before it, and wait
// for it before they read or write.
template <typename... KA, typename... A>
cudaError_t launch(void (*k)(KA...), int grid, bool dep, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(UT);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = dep;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// The sums of squares of the whole list; blocks: how many.
template <int N>
cudaError_t launch_squares(const rnnt_grad_list* l, const void* const* grads, double* part,
                           int* blocks, int* launches, cudaStream_t st) {
  static std::atomic<int> known[kDeviceSlots];
  int most = 0, i = 0;
  cudaError_t e = resident(k_clip_squares<N>, known, &most);
  *blocks = 0;
  *launches = 0;
  do {
    NormTable<N> t;
    i = next_chunks(l, i, &t.c, [&](int k, int j) {
      t.g[k] = grads[j];
      return head_of(grads[j], t.c.bf16[k]);
    });
    // (every launch of a call fills the same sums)
    if (!*launches)
      *blocks = std::min({PARTS, most, i < l->n ? PARTS : std::max(1, t.c.first[t.c.n])});
    if (e == cudaSuccess) e = launch(k_clip_squares<N>, *blocks, false, st, t, part, *launches > 0);
    if (e != cudaSuccess) return e;
    ++*launches;
  } while (i < l->n);
  return e;
}

template <int N>
cudaError_t launch_scale(const rnnt_grad_list* l, const void* const* grads, void* const* into,
                         NormArgs a, int* launches, cudaStream_t st) {
  static std::atomic<int> known[kDeviceSlots];
  int most = 0;
  cudaError_t e = resident(k_clip_scale<N>, known, &most);
  for (int i = 0; i < l->n && e == cudaSuccess;) {
    ScaleTable<N> t;
    i = next_chunks(l, i, &t.c, [&](int k, int j) {
      t.g[k] = grads[j];
      t.into[k] = into[j];
      const int h = head_of(grads[j], t.c.bf16[k]);
      t.alike[k] = h == head_of(into[j], t.c.bf16[k]);
      return h;
    });
    if (!t.c.n) break;
    // (only the first may start under the squares: a later one's tail says nothing of them)
    e = launch(k_clip_scale<N>, std::min(most, t.c.first[t.c.n]), *launches == 0, st, t, a);
    a.n = 0;
    ++*launches;
  }
  return e;
}

// The whole call.  (So few chunks are of as few tensors, and all of them have one.)
cudaError_t launch_short(const rnnt_grad_list* l, const void* const* grads, void* const* into,
                         float max_norm, float eps, float* clip, cudaStream_t st) {
  static std::atomic<bool> known[kDeviceSlots];
  ScaleTable<SHORT> t;
  t.into[0] = nullptr;
  next_chunks(l, 0, &t.c, [&](int k, int j) {
    t.g[k] = grads[j];
    t.into[k] = into ? into[j] : nullptr;
    const int h = head_of(grads[j], t.c.bf16[k]);
    t.alike[k] = into && h == head_of(into[j], t.c.bf16[k]);
    return h;
  });
  std::atomic<bool>& d = known[device_slot()];
  if (!d.load()) {
    const cudaError_t e = cudaFuncSetAttribute(
        k_clip_short, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    d.store(true);
  }
  int blocks = 1;
  while (blocks * CGROUPS < t.c.first[t.c.n]) blocks *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(UT * CGROUPS);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_clip_short, t, max_norm, eps, clip);
}

struct AdamLists {
  float* const* p;
  const void* const* g;
  float* const* m;
  float* const* v;
  void* const* low;
};

// The next launch of up to N of the list's tensors from *i on, of `left` with elements.
template <int N>
cudaError_t launch_adamw(const rnnt_grad_list* l, const rnnt_adamw_opts* o, const AdamLists& x,
                         AdamArgs a, int* i, int* left, cudaStream_t st) {
  static std::atomic<int> known[kDeviceSlots];
  int most = 0;
  const cudaError_t e = resident(k_adamw<N>, known, &most);
  if (e != cudaSuccess) return e;
  AdamTable<N> t;
  *i = next_chunks(l, *i, &t.c, [&](int k, int j) {
    t.g[k] = x.g[j];
    t.p[k] = x.p[j];
    t.m[k] = x.m[j];
    t.v[k] = x.v[j];
    t.low[k] = x.low ? (__nv_bfloat16*)x.low[j] : nullptr;
    t.decay[k] = o->decays ? o->decays[j] : o->decay;
    const int h = head_of(x.g[j], t.c.bf16[k]);
    const bool alike = h == head_of(x.p[j], false) && h == head_of(x.m[j], false) &&
                       h == head_of(x.v[j], false) && (!t.low[k] || h == head_of(t.low[k], true));
    return alike ? h : -1;
  });
  *left -= t.c.n;
  a.last = *left == 0;
  return launch(k_adamw<N>, std::min(most, t.c.first[t.c.n]), true, st, t, a);
}

}  // namespace
}  // namespace rnnt

using namespace rnnt;

extern "C" {

size_t rnnt_clip_workspace_bytes(const rnnt_grad_list* list) {
  return list_ok(list) ? align_up(PARTS * sizeof(double)) : 0;
}

rnnt_status rnnt_clip(const rnnt_grad_list* list, const void* const* grads, void* const* into,
                      float max_norm, float eps, float* clip, void* ws, size_t ws_bytes,
                      rnnt_stream stream) {
  if (!list_ok(list) || !clip || !ws || !aligned_to(clip, 4) || !aligned_to(ws, ALIGN))
    return RNNT_ERR_INVALID_ARG;
  if (!(max_norm >= 0.f) || !(eps >= 0.f) || !isfinite(eps) || (max_norm == 0.f && eps == 0.f))
    return RNNT_ERR_INVALID_ARG;
  if (!pointers_ok(list, grads, true) ||
      (into && !pointers_ok(list, (const void* const*)into, true)))
    return RNNT_ERR_INVALID_ARG;
  if (ws_bytes < rnnt_clip_workspace_bytes(list)) return RNNT_ERR_WORKSPACE_TOO_SMALL;
  if (into) {
    Spans s(2 * (size_t)list->n);
    if (!s.ok()) return RNNT_ERR_CUDA;
    auto bytes = [&](int i) { return (size_t)list->count[i] * (is_bf16(list, i) ? 2 : 4); };
    s.add(list->n, true, [&](int i) { return into[i]; }, bytes);
    s.add(list->n, false, [&](int i) { return grads[i] != into[i] ? grads[i] : nullptr; }, bytes);
    if (s.overlap()) return RNNT_ERR_INVALID_ARG;
  }
  cudaStream_t st = (cudaStream_t)stream;
  double* part = (double*)ws;
  const bool few = list->n <= FEW;
  long long chunks = 0;
  for (int i = 0; i < list->n; ++i) chunks += cdiv(list->count[i], CHUNK);
  if (chunks <= SHORT) {
    OPS_LAUNCH("clip_norm", launch_short(list, grads, into, max_norm, eps, clip, st));
    return RNNT_OK;
  }
  NormArgs a{part, 0, max_norm, eps, clip};
  {
    ProfScope ps("clip_norm", st);
    int launches = 0;
    OPS_CHECK((few ? launch_squares<FEW>(list, grads, part, &a.n, &launches, st)
                   : launch_squares<MANY>(list, grads, part, &a.n, &launches, st)));
    if (!into) {
      OPS_CHECK(launch(k_clip_norm, 1, true, st, a));
      ++launches;
    }
    ps.set_kernels(launches);
  }
  if (!into) return RNNT_OK;
  ProfScope ps("clip_scale", st);
  int launches = 0;
  OPS_CHECK((few ? launch_scale<FEW>(list, grads, into, a, &launches, st)
                 : launch_scale<MANY>(list, grads, into, a, &launches, st)));
  ps.set_kernels(launches);
  return RNNT_OK;
}

rnnt_status rnnt_adamw(const rnnt_grad_list* list, const rnnt_adamw_opts* o,
                       float* const* params, const void* const* grads, float* const* m,
                       float* const* v, void* const* low, const float* lr, const float* clip,
                       int32_t* steps, rnnt_stream stream) {
  if (!list_ok(list) || !o || !steps || !aligned_to(steps, 4) || !aligned_to(lr, 4) ||
      !aligned_to(clip, 4))
    return RNNT_ERR_INVALID_ARG;
  if (!(o->beta1 >= 0 && o->beta1 < 1 && o->beta2 >= 0 && o->beta2 < 1) || !(o->eps >= 0.f) ||
      !isfinite(o->eps) || (!lr && !isfinite(o->lr)))
    return RNNT_ERR_INVALID_ARG;
  if (!pointers_ok(list, (const void* const*)params, false) || !pointers_ok(list, grads, true) ||
      !pointers_ok(list, (const void* const*)m, false) ||
      !pointers_ok(list, (const void* const*)v, false))
    return RNNT_ERR_INVALID_ARG;
  for (int i = 0; i < list->n; ++i) {
    if (low && list->count[i] && !aligned_to(low[i], 2)) return RNNT_ERR_INVALID_ARG;
    if (!isfinite(o->decays ? o->decays[i] : o->decay)) return RNNT_ERR_INVALID_ARG;
  }
  {
    Spans s(5 * (size_t)list->n);
    if (!s.ok()) return RNNT_ERR_CUDA;
    auto fp32 = [&](int i) { return (size_t)list->count[i] * 4; };
    for (float* const* x : {params, m, v})
      s.add(list->n, true, [&](int i) { return x[i]; }, fp32);
    if (low)
      s.add(list->n, true, [&](int i) { return low[i]; }, [&](int i) { return fp32(i) / 2; });
    s.add(list->n, false, [&](int i) { return grads[i]; },
          [&](int i) { return fp32(i) / (is_bf16(list, i) ? 2 : 1); });
    if (s.overlap()) return RNNT_ERR_INVALID_ARG;
  }
  cudaStream_t st = (cudaStream_t)stream;
  AdamArgs a{};
  a.b1 = (float)o->beta1; a.b2 = (float)o->beta2;
  a.nb1 = (float)(1 - o->beta1); a.nb2 = (float)(1 - o->beta2);
  a.log1 = (float)log(o->beta1); a.log2 = (float)log(o->beta2);
  a.eps = o->eps; a.lr = o->lr;
  a.lr_dev = lr; a.clip = clip; a.steps = steps;
  ProfScope ps("adamw", st);
  int launches = 0;
  const AdamLists x{params, grads, m, v, low};
  int left = 0;
  for (int i = 0; i < list->n; ++i) left += list->count[i] > 0;
  for (int i = 0; left > 0; ++launches)
    OPS_CHECK((list->n <= FEW ? launch_adamw<FEW>(list, o, x, a, &i, &left, st)
                              : launch_adamw<MANY>(list, o, x, a, &i, &left, st)));
  ps.set_kernels(launches);
  return RNNT_OK;
}

int rnnt_testing_overlap(int n, const void* const* p, const size_t* bytes, const int* written) {
  Spans s(n);
  if (!s.ok()) return -1;
  for (int i = 0, end; i < n; i = end) {  // lists: pieces of one kind
    for (end = i; end < n && !written[end] == !written[i];) ++end;
    s.add(end - i, written[i] != 0, [&](int k) { return p[i + k]; },
          [&](int k) { return bytes[i + k]; });
  }
  return s.overlap();
}

}  // extern "C"
