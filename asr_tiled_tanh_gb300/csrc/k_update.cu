// k_update.cu -- gradient clipping and the AdamW update over lists of tensors
// (include/rnnt_ops.h).
#include <algorithm>
#include <new>

#include "ops.h"
#include "ptx.cuh"

namespace rnnt {
namespace {

constexpr int UT = 256;       // threads
constexpr int CHUNK = 2048;   // elements of one tensor that a block takes at a time
constexpr int TENSORS = 64;   // tensors a launch (its tables are kernel parameters)
constexpr int PARTS = 1024;   // sums of squares that the workspace holds

// A launch's tensors, cut into chunks that are numbered through.
struct Chunks {
  int n;
  int first[TENSORS + 1];  // chunks before each tensor
  long long count[TENSORS];
  uint8_t bf16[TENSORS];   // the gradient's type
};

// Tensor of chunk k < first[n] (the last one that begins at or before it: tensors
// of no elements begin where the next one does).
__device__ __forceinline__ int tensor_of(const Chunks& c, int k) {
  int lo = 0, hi = c.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.first[mid] <= k) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float grad_at(const void* g, bool bf16, long long i) {
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

struct NormTable {
  Chunks c;
  const void* g[TENSORS];
};

// part[block]: the block's sum of squares (added to what an earlier launch of the
// same call left there).
__global__ void __launch_bounds__(UT)
k_clip_squares(const __grid_constant__ NormTable t, double* __restrict__ part, int add) {
  __shared__ double scr[UT / 32];
  double sum = 0;
  for (int k = blockIdx.x; k < t.c.first[t.c.n]; k += gridDim.x) {
    const int i = tensor_of(t.c, k);
    const long long at = (long long)(k - t.c.first[i]) * CHUNK;
    const int n = (int)min((long long)CHUNK, t.c.count[i] - at);
    for (int e = threadIdx.x; e < n; e += UT) {
      const double g = grad_at(t.g[i], t.c.bf16[i], at + e);
      sum += g * g;
    }
  }
  sum = block_sum(sum, scr);
  if (threadIdx.x == 0) part[blockIdx.x] = add ? part[blockIdx.x] + sum : sum;
}

__global__ void __launch_bounds__(UT)
k_clip_norm(const double* __restrict__ part, int n, float max_norm, float eps,
            float* __restrict__ clip) {
  __shared__ double scr[UT / 32];
  double sum = 0;
  for (int k = threadIdx.x; k < n; k += UT) sum += part[k];
  sum = block_sum(sum, scr);
  if (threadIdx.x == 0) {
    const double norm = sqrt(sum), q = (double)max_norm / (norm + (double)eps);
    clip[0] = (float)norm;
    clip[1] = q >= 1 ? 1.f : (float)q;  // (NaN stays)
  }
}

struct ScaleTable {
  Chunks c;
  const void* g[TENSORS];
  void* into[TENSORS];
};

__global__ void __launch_bounds__(UT)
k_clip_scale(const __grid_constant__ ScaleTable t, const float* __restrict__ clip) {
  const float s = clip[1];
  const int k = blockIdx.x, i = tensor_of(t.c, k);
  if (s == 1.f && t.g[i] == t.into[i]) return;
  const long long at = (long long)(k - t.c.first[i]) * CHUNK;
  const int n = (int)min((long long)CHUNK, t.c.count[i] - at);
  for (int e = threadIdx.x; e < n; e += UT) {
    const float v = s * grad_at(t.g[i], t.c.bf16[i], at + e);
    if (t.c.bf16[i]) ((__nv_bfloat16*)t.into[i])[at + e] = __float2bfloat16_rn(v);
    else ((float*)t.into[i])[at + e] = v;
  }
}

struct AdamTable {
  Chunks c;
  const void* g[TENSORS];
  float *p[TENSORS], *m[TENSORS], *v[TENSORS];
  __nv_bfloat16* low[TENSORS];
  float decay[TENSORS];
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

__global__ void __launch_bounds__(UT)
k_adamw(const __grid_constant__ AdamTable t, AdamArgs a) {
  const int done = a.steps[0];
  const float scale = a.clip ? a.clip[1] : 1.f;
  const bool take = !a.clip || isfinite(a.clip[0]);
  if (take) {
    const float lr = a.lr_dev ? *a.lr_dev : a.lr;
    // 1 - beta^t without the cancellation
    const float c1 = -expm1f((float)(done + 1) * a.log1), c2 = -expm1f((float)(done + 1) * a.log2);
    const int k = blockIdx.x, i = tensor_of(t.c, k);
    const long long at = (long long)(k - t.c.first[i]) * CHUNK;
    const int n = (int)min((long long)CHUNK, t.c.count[i] - at);
    for (int e = threadIdx.x; e < n; e += UT) {
      const float g = scale * grad_at(t.g[i], t.c.bf16[i], at + e);
      const float m = fmaf(a.b1, t.m[i][at + e], a.nb1 * g);
      const float v = fmaf(a.b2, t.v[i][at + e], a.nb2 * g * g);
      float p = t.p[i][at + e];
      p -= lr * fmaf(t.decay[i], p, (m / c1) / (sqrtf(v / c2) + a.eps));
      t.m[i][at + e] = m;
      t.v[i][at + e] = v;
      t.p[i][at + e] = p;
      if (t.low[i]) t.low[i][at + e] = __float2bfloat16_rn(p);
    }
  }
  // the last block to come here, when every block has read the count, counts the
  // update, and the second word wraps to 0
  __syncthreads();
  if (threadIdx.x == 0 && atomicInc((unsigned*)a.steps + 1, gridDim.x - 1) == gridDim.x - 1 &&
      a.last && take)
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

// The next launch's tensors, from i on, into c; fill(k, j): tensor j is its k-th.
// Returns the tensor after them.
template <typename F>
int next_chunks(const rnnt_grad_list* l, int i, Chunks* c, F fill) {
  c->n = 0;
  c->first[0] = 0;
  for (; i < l->n && c->n < TENSORS; ++i) {
    if (!l->count[i]) continue;
    const long long chunks = cdiv(l->count[i], CHUNK);
    if (c->n && c->first[c->n] + chunks > 0x7fffffff) break;
    const int k = c->n++;
    c->count[k] = l->count[i];
    c->bf16[k] = is_bf16(l, i);
    c->first[k + 1] = c->first[k] + (int)chunks;
    fill(k, i);
  }
  return i;
}

int norm_blocks() { return std::min(PARTS, 4 * num_sms()); }

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
  const int blocks = norm_blocks();
  {
    ProfScope ps("clip_norm", st);
    int launches = 1, i = 0;
    do {
      NormTable t;
      i = next_chunks(list, i, &t.c, [&](int k, int j) { t.g[k] = grads[j]; });
      k_clip_squares<<<blocks, UT, 0, st>>>(t, part, launches > 1);
      OPS_CHECK(cudaGetLastError());
      ++launches;
    } while (i < list->n);
    k_clip_norm<<<1, UT, 0, st>>>(part, blocks, max_norm, eps, clip);
    OPS_CHECK(cudaGetLastError());
    ps.set_kernels(launches);
  }
  if (!into) return RNNT_OK;
  ProfScope ps("clip_scale", st);
  int launches = 0;
  for (int i = 0; i < list->n;) {
    ScaleTable t;
    i = next_chunks(list, i, &t.c, [&](int k, int j) {
      t.g[k] = grads[j];
      t.into[k] = into[j];
    });
    if (!t.c.n) break;
    k_clip_scale<<<t.c.first[t.c.n], UT, 0, st>>>(t, clip);
    OPS_CHECK(cudaGetLastError());
    ++launches;
  }
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
  int launches = 0, left = 0;
  for (int i = 0; i < list->n; ++i) left += list->count[i] > 0;
  for (int i = 0; left > 0;) {
    AdamTable t;
    i = next_chunks(list, i, &t.c, [&](int k, int j) {
      t.g[k] = grads[j];
      t.p[k] = params[j];
      t.m[k] = m[j];
      t.v[k] = v[j];
      t.low[k] = low ? (__nv_bfloat16*)low[j] : nullptr;
      t.decay[k] = o->decays ? o->decays[j] : o->decay;
    });
    left -= t.c.n;
    a.last = left == 0;
    k_adamw<<<t.c.first[t.c.n], UT, 0, st>>>(t, a);
    OPS_CHECK(cudaGetLastError());
    ++launches;
  }
  ps.set_kernels(launches);
  return RNNT_OK;
}

}  // extern "C"
