// k_update.cu -- gradient clipping and the AdamW update over lists of tensors
// (include/rnnt_ops.h).
#include <algorithm>
#include <atomic>
#include <new>

#include "ops.h"
#include "ptx.cuh"

namespace rnnt {
namespace {

constexpr int UT = 256;       // threads
constexpr int CHUNK = 8192;   // elements of one tensor that a block takes at a time
constexpr int PARTS = 1024;   // sums of squares that the workspace holds
// Tensors a launch: its tables are kernel parameters, of which there are 32 KB.
constexpr int FEW = 32, MANY = 512;

// A launch's tensors, cut into chunks that are numbered through.
template <int N>
struct Chunks {
  int n;
  int first[N + 1];  // chunks before each tensor
  long long count[N];
  uint8_t bf16[N];   // the gradient's type
  uint8_t vec[N];    // every tensor of the place is aligned to four elements
};

// Tensor of chunk k < first[n] (the last one that begins at or before it), and the
// chunk's elements.
struct Piece {
  int i, n;
  long long at;
};
template <int N>
__device__ __forceinline__ Piece piece_of(const Chunks<N>& c, int k) {
  int lo = 0, hi = c.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.first[mid] <= k) lo = mid;
    else hi = mid - 1;
  }
  Piece p;
  p.i = lo;
  p.at = (long long)(k - c.first[lo]) * CHUNK;
  p.n = (int)min((long long)CHUNK, c.count[lo] - p.at);
  return p;
}

// Four elements, or one, as they are stored and widened.
__device__ __forceinline__ float4 widen4(uint2 u) {
  return make_float4(ptx::bf16lo(u.x), ptx::bf16hi(u.x), ptx::bf16lo(u.y), ptx::bf16hi(u.y));
}
__device__ __forceinline__ float4 grad4(const void* g, bool bf16, long long i) {
  return bf16 ? widen4(*(const uint2*)((const __nv_bfloat16*)g + i)) : *(const float4*)((const float*)g + i);
}
__device__ __forceinline__ float grad1(const void* g, bool bf16, long long i) {
  return bf16 ? __bfloat162float(((const __nv_bfloat16*)g)[i]) : ((const float*)g)[i];
}

// Sum of v over the block's threads in a fixed order, for thread 0.
__device__ __forceinline__ double block_sum(double v, double* scr) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) scr[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int k = 1; k < UT / 32; ++k) v += scr[k];
  return v;
}

// ---- norm -------------------------------------------------------------------------
// A thread's 32 elements of a chunk: squares added in fp32 (33 roundings of terms of
// one sign), in fp64 where that left the range or came near its bottom.  fp64 for
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
  double d = 0;
#pragma unroll 4
  for (int k = 0; k < EACH; ++k) d = fma((double)g[k], (double)g[k], d);
  return d;
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
  for (int k = blockIdx.x; k < t.c.first[t.c.n]; k += gridDim.x) {
    const Piece p = piece_of(t.c, k);
    const bool bf16 = t.c.bf16[p.i];
    const void* g = t.g[p.i];
    float v[EACH];
    if (t.c.vec[p.i]) {
      const int whole = p.n & ~3;
#pragma unroll
      for (int j = 0; j < EACH / 4; ++j) {
        const int e = (j * UT + threadIdx.x) * 4;
        float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < whole) {
          q = grad4(g, bf16, p.at + e);
        } else if (e < p.n) {  // the tensor's last one to three
          q.x = grad1(g, bf16, p.at + e);
          if (e + 1 < p.n) q.y = grad1(g, bf16, p.at + e + 1);
          if (e + 2 < p.n) q.z = grad1(g, bf16, p.at + e + 2);
        }
        v[4 * j] = q.x;
        v[4 * j + 1] = q.y;
        v[4 * j + 2] = q.z;
        v[4 * j + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        const int e = j * UT + threadIdx.x;
        v[j] = e < p.n ? grad1(g, bf16, p.at + e) : 0.f;
      }
    }
    sum += squares(v);
  }
  sum = block_sum(sum, scr);
  if (threadIdx.x == 0) part[blockIdx.x] = add ? part[blockIdx.x] + sum : sum;
}

__global__ void __launch_bounds__(UT)
k_clip_norm(const double* __restrict__ part, int n, float max_norm, float eps,
            float* __restrict__ clip) {
  __shared__ double scr[UT / 32];
  ptx::griddep_launch();
  ptx::griddep_wait();
  double sum = 0;
#pragma unroll
  for (int k = 0; k < PARTS / UT; ++k)
    if (threadIdx.x + k * UT < n) sum += __ldcg(part + threadIdx.x + k * UT);
  sum = block_sum(sum, scr);
  if (threadIdx.x == 0) {
    const double norm = sqrt(sum), q = (double)max_norm / (norm + (double)eps);
    clip[0] = (float)norm;
    clip[1] = q >= 1 ? 1.f : (float)q;  // (NaN stays)
  }
}

// ---- scaling ----------------------------------------------------------------------
template <int N>
struct ScaleTable {
  Chunks<N> c;
  const void* g[N];
  void* into[N];
};

// (Chunks are taken from the end: the norm's pass left those in L2.)
template <int N>
__global__ void __launch_bounds__(UT)
k_clip_scale(const __grid_constant__ ScaleTable<N> t, const float* clip) {
  ptx::griddep_wait();
  const float s = __ldcg(clip + 1);
#pragma unroll 1
  for (int k = t.c.first[t.c.n] - 1 - blockIdx.x; k >= 0; k -= gridDim.x) {
    const Piece p = piece_of(t.c, k);
    const bool bf16 = t.c.bf16[p.i];
    const void* g = t.g[p.i];
    void* into = t.into[p.i];
    if (s == 1.f && g == into) continue;
    int done = 0;
    if (t.c.vec[p.i]) {
      done = p.n & ~3;
#pragma unroll
      for (int j = 0; j < EACH / 4; ++j) {
        const int e = (j * UT + threadIdx.x) * 4;
        if (e >= done) continue;
        const float4 q = grad4(g, bf16, p.at + e);
        if (bf16)
          *(uint2*)((__nv_bfloat16*)into + p.at + e) =
              make_uint2(ptx::pack_bf16x2(s * q.x, s * q.y), ptx::pack_bf16x2(s * q.z, s * q.w));
        else
          *(float4*)((float*)into + p.at + e) = make_float4(s * q.x, s * q.y, s * q.z, s * q.w);
      }
    }
#pragma unroll 8
    for (int e = done + threadIdx.x; e < p.n; e += UT) {
      const float v = s * grad1(g, bf16, p.at + e);
      if (bf16) ((__nv_bfloat16*)into)[p.at + e] = __float2bfloat16_rn(v);
      else ((float*)into)[p.at + e] = v;
    }
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

// Bound by DRAM: 28 to 30 bytes an element in 8 streams.
template <int N>
__global__ void __launch_bounds__(UT)
k_adamw(const __grid_constant__ AdamTable<N> t, AdamArgs a) {
  ptx::griddep_wait();
  const int done = __ldcg(a.steps);
  const bool take = !a.clip || isfinite(__ldcg(a.clip));
  if (take) {
    AdamStep f;
    f.b1 = a.b1; f.b2 = a.b2; f.nb1 = a.nb1; f.nb2 = a.nb2; f.eps = a.eps;
    f.scale = a.clip ? __ldcg(a.clip + 1) : 1.f;
    f.lr = a.lr_dev ? __ldcg(a.lr_dev) : a.lr;
    // 1 - beta^t without the cancellation
    f.r1 = 1.f / -expm1f((float)(done + 1) * a.log1);
    f.r2 = 1.f / -expm1f((float)(done + 1) * a.log2);
#pragma unroll 1
    for (int k = t.c.first[t.c.n] - 1 - blockIdx.x; k >= 0; k -= gridDim.x) {
      const Piece c = piece_of(t.c, k);
      const bool bf16 = t.c.bf16[c.i];
      const void* g = t.g[c.i];
      float *p = t.p[c.i] + c.at, *m = t.m[c.i] + c.at, *v = t.v[c.i] + c.at;
      __nv_bfloat16* low = t.low[c.i];
      if (low) low += c.at;
      f.decay = t.decay[c.i];
      int vec = 0;
      if (t.c.vec[c.i]) {
        vec = c.n & ~3;
#pragma unroll 2
        for (int e = threadIdx.x * 4; e < vec; e += UT * 4) {
          const float4 gq = grad4(g, bf16, c.at + e);
          float4 pq = *(const float4*)(p + e), mq = *(const float4*)(m + e),
                 vq = *(const float4*)(v + e);
          f(pq, mq, vq, gq);
          *(float4*)(p + e) = pq;
          *(float4*)(m + e) = mq;
          *(float4*)(v + e) = vq;
          if (low)
            *(uint2*)(low + e) =
                make_uint2(ptx::pack_bf16x2(pq.x, pq.y), ptx::pack_bf16x2(pq.z, pq.w));
        }
      }
#pragma unroll 2
      for (int e = vec + threadIdx.x; e < c.n; e += UT) {
        float pe = p[e], me = m[e], ve = v[e];
        f(pe, me, ve, grad1(g, bf16, c.at + e));
        p[e] = pe;
        m[e] = me;
        v[e] = ve;
        if (low) low[e] = __float2bfloat16_rn(pe);
      }
    }
  }
  // The last block to come here counts the update, when every block has read the
  // count, and the second word wraps to 0.
  __syncthreads();
  if (threadIdx.x) return;
  __threadfence();
  if (atomicInc((unsigned*)a.steps + 1, gridDim.x - 1) == gridDim.x - 1 && a.last && take)
    a.steps[0] = done + 1;
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

// Memory that a call writes, and what must stay clear of it.
struct Span {
  uintptr_t from, to;
  bool written;
};
struct Spans {
  Span* s;
  size_t n = 0;
  bool sorted = true;
  explicit Spans(size_t most) : s(new (std::nothrow) Span[most ? most : 1]) {}
  ~Spans() { delete[] s; }
  void add(const void* p, size_t bytes, bool written) {
    if (!p || !bytes) return;
    s[n++] = {(uintptr_t)p, (uintptr_t)p + bytes, written};
    if (n > 1 && s[n - 1].from < s[n - 2].from) sorted = false;
  }
  // whether a written one meets another
  bool overlap() {
    if (!sorted)
      std::sort(s, s + n, [](const Span& a, const Span& b) { return a.from < b.from; });
    uintptr_t read_to = 0, written_to = 0;
    for (size_t i = 0; i < n; ++i) {
      if (s[i].from < written_to || (s[i].written && s[i].from < read_to)) return true;
      uintptr_t& to = s[i].written ? written_to : read_to;
      to = std::max(to, s[i].to);
    }
    return false;
  }
};

// The next launch's tensors, from i on, into c; fill(k, j): tensor j is its k-th,
// and returns whether its places are aligned to four elements.  Returns the tensor
// after them.
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
    c->vec[k] = fill(k, i);
  }
  return i;
}

// Aligned to four elements of fp32, or of bf16.
bool quads(const void* p, bool bf16) { return aligned_to(p, bf16 ? 8 : 16); }

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
      return quads(grads[j], t.c.bf16[k]);
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
                         const float* clip, int* launches, cudaStream_t st) {
  static std::atomic<int> known[kDeviceSlots];
  int most = 0;
  cudaError_t e = resident(k_clip_scale<N>, known, &most);
  for (int i = 0; i < l->n && e == cudaSuccess;) {
    ScaleTable<N> t;
    i = next_chunks(l, i, &t.c, [&](int k, int j) {
      t.g[k] = grads[j];
      t.into[k] = into[j];
      return quads(grads[j], t.c.bf16[k]) && quads(into[j], t.c.bf16[k]);
    });
    if (!t.c.n) break;
    // (only the first may start under the norm: a later one's tail says nothing of it)
    e = launch(k_clip_scale<N>, std::min(most, t.c.first[t.c.n]), *launches == 0, st, t, clip);
    ++*launches;
  }
  return e;
}

struct AdamLists {
  float* const* p;
  const void* const* g;
  float* const* m;
  float* const* v;
  void* const* low;
};

template <int N>
cudaError_t launch_adamw(const rnnt_grad_list* l, const rnnt_adamw_opts* o, const AdamLists& x,
                         AdamArgs a, int* launches, cudaStream_t st) {
  static std::atomic<int> known[kDeviceSlots];
  int most = 0, left = 0;
  cudaError_t e = resident(k_adamw<N>, known, &most);
  for (int i = 0; i < l->n; ++i) left += l->count[i] > 0;
  for (int i = 0; left > 0 && e == cudaSuccess;) {
    AdamTable<N> t;
    i = next_chunks(l, i, &t.c, [&](int k, int j) {
      t.g[k] = x.g[j];
      t.p[k] = x.p[j];
      t.m[k] = x.m[j];
      t.v[k] = x.v[j];
      t.low[k] = x.low ? (__nv_bfloat16*)x.low[j] : nullptr;
      t.decay[k] = o->decays ? o->decays[j] : o->decay;
      return quads(x.g[j], t.c.bf16[k]) && quads(x.p[j], false) && quads(x.m[j], false) &&
             quads(x.v[j], false) && quads(t.low[k], true);
    });
    left -= t.c.n;
    a.last = left == 0;
    e = launch(k_adamw<N>, std::min(most, t.c.first[t.c.n]), *launches == 0, st, t, a);
    ++*launches;
  }
  return e;
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
    if (!s.s) return RNNT_ERR_CUDA;
    for (int i = 0; i < list->n; ++i) {
      const size_t bytes = list->count[i] * (is_bf16(list, i) ? 2 : 4);
      s.add(into[i], bytes, true);
      if (grads[i] != into[i]) s.add(grads[i], bytes, false);
    }
    if (s.overlap()) return RNNT_ERR_INVALID_ARG;
  }
  cudaStream_t st = (cudaStream_t)stream;
  double* part = (double*)ws;
  const bool few = list->n <= FEW;
  {
    ProfScope ps("clip_norm", st);
    int blocks = 0, launches = 0;
    OPS_CHECK((few ? launch_squares<FEW>(list, grads, part, &blocks, &launches, st)
                   : launch_squares<MANY>(list, grads, part, &blocks, &launches, st)));
    OPS_CHECK(launch(k_clip_norm, 1, true, st, part, blocks, max_norm, eps, clip));
    ps.set_kernels(launches + 1);
  }
  if (!into) return RNNT_OK;
  ProfScope ps("clip_scale", st);
  int launches = 0;
  OPS_CHECK((few ? launch_scale<FEW>(list, grads, into, clip, &launches, st)
                 : launch_scale<MANY>(list, grads, into, clip, &launches, st)));
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
    if (!s.s) return RNNT_ERR_CUDA;
    for (int i = 0; i < list->n; ++i) s.add(params[i], 4 * list->count[i], true);
    for (int i = 0; i < list->n; ++i) s.add(m[i], 4 * list->count[i], true);
    for (int i = 0; i < list->n; ++i) s.add(v[i], 4 * list->count[i], true);
    for (int i = 0; low && i < list->n; ++i) s.add(low[i], 2 * list->count[i], true);
    for (int i = 0; i < list->n; ++i)
      s.add(grads[i], (is_bf16(list, i) ? 2 : 4) * list->count[i], false);
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
  OPS_CHECK((list->n <= FEW ? launch_adamw<FEW>(list, o, x, a, &launches, st)
                            : launch_adamw<MANY>(list, o, x, a, &launches, st)));
  ps.set_kernels(launches);
  return RNNT_OK;
}

}  // extern "C"
