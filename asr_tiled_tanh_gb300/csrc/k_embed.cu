// k_embed.cu -- the prediction network's label embedding (include/rnnt_ops.h).
#include <atomic>

#include "ops.h"
#include "ptx.cuh"

namespace rnnt {
namespace {

struct EmbedArgs {
  int B, U1, V, D, blank, sos;
  float scale;
  long long ld_table, ld_rows;
  const int32_t* ids;
  const int32_t* U_len;
  int32_t* status;
};

// Label of row n = (b, u); -1 for a row that does not exist or whose label is
// out of range (both are recorded).
__device__ __forceinline__ int label_of(const EmbedArgs& a, int n) {
  const int b = n / a.U1, u = n - b * a.U1;
  if (a.U_len) {
    const int ul = __ldg(a.U_len + b);
    if (ul < 0 || ul >= a.U1) {
      report(a.status, RNNT_ERR_LENGTH_RANGE);
      return -1;
    }
    if (u > ul) return -1;
  }
  if (a.sos && u == 0) return a.blank;
  const int id = __ldg(a.ids + n);
  if (id < 0 || id >= a.V) {
    report(a.status, RNNT_ERR_LABEL_RANGE);
    return -1;
  }
  return id;
}

// ---- rows -------------------------------------------------------------------
// hL row n = scale * E[label].  Bound by its stores (a row is written once, the
// table's rows come from L2).  A lane owns VEC consecutive columns: eight on
// 16-byte aligned rows, else two or one.
//
// A lane's VEC elements as they are loaded (the registers that loads in flight
// hold), and widened.
template <int BYTES> struct RawWord;
template <> struct RawWord<2> { using type = unsigned short; };
template <> struct RawWord<4> { using type = unsigned int; };
template <> struct RawWord<8> { using type = uint2; };
template <> struct RawWord<16> { using type = uint4; };

template <int VEC, typename T>
struct Raw {
  static constexpr int BYTES = VEC * sizeof(T), WORDS = BYTES > 16 ? BYTES / 16 : 1;
  using W = typename RawWord<(BYTES > 16 ? 16 : BYTES)>::type;
  W w[WORDS];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = W{};
  }
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = __ldg((const W*)p + i);
  }
  // data that an earlier kernel may still write when this one starts: not by the
  // read-only path, which holds for what stays unchanged while a kernel runs
  __device__ __forceinline__ void load_late(const T* p) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = __ldcg((const W*)p + i);
  }
  __device__ __forceinline__ void widen(float (&v)[VEC]) const {
    if constexpr (sizeof(T) == 4) {
      const uint32_t* u = (const uint32_t*)w;
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = __uint_as_float(u[i]);
    } else if constexpr (VEC == 1) {
      v[0] = __uint_as_float((uint32_t)w[0] << 16);
    } else {
      const uint32_t* u = (const uint32_t*)w;
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        v[2 * i] = ptx::bf16lo(u[i]);
        v[2 * i + 1] = ptx::bf16hi(u[i]);
      }
    }
  }
};

template <int VEC>
__device__ __forceinline__ void scale_vec(float (&v)[VEC], float s) {
  if constexpr (VEC == 1) {
    v[0] *= s;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      const float2 x = __fmul2_rn(make_float2(v[i], v[i + 1]), make_float2(s, s));
      v[i] = x.x;
      v[i + 1] = x.y;
    }
  }
}
template <int VEC>
__device__ __forceinline__ void add_vec(float (&a)[VEC], const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    a[0] += v[0];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      const float2 x = __fadd2_rn(make_float2(a[i], a[i + 1]), make_float2(v[i], v[i + 1]));
      a[i] = x.x;
      a[i + 1] = x.y;
    }
  }
}

// (16-byte stores say that they stream: the rows of a large batch would else
// push one another's lines out half written, 23 against 19 us for 106 MB)
template <int VEC, typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    *p = from_f<T>(v[0]);
  } else if constexpr (VEC == 2 && sizeof(T) == 4) {
    *(float2*)p = make_float2(v[0], v[1]);
  } else if constexpr (VEC == 2) {
    *(uint32_t*)p = ptx::pack_bf16x2(v[0], v[1]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4)
      __stcs((float4*)(p + i), make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
  } else {
    __stcs((uint4*)p, make_uint4(ptx::pack_bf16x2(v[0], v[1]), ptx::pack_bf16x2(v[2], v[3]),
                                 ptx::pack_bf16x2(v[4], v[5]), ptx::pack_bf16x2(v[6], v[7])));
  }
}

constexpr int ROWS_THREADS = 128;

// A warp writes K steps of 32 / (1 << lg) rows, 1 << lg lanes to a row.  Each
// lane looks one row's label up; the rows take theirs by shuffle.
template <int VEC, int K, typename TE, typename TR>
__global__ void __launch_bounds__(ROWS_THREADS)
k_embed_rows(EmbedArgs a, int lg, const TE* __restrict__ table, TR* __restrict__ rows) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vpr = a.D / VEC, per = 32 >> lg;
  const long long n0 = ((long long)blockIdx.x * (ROWS_THREADS / 32) + warp) * (K * per);
  const int N = a.B * a.U1;
  const int left = (int)max(0LL, min((long long)(K * per), N - n0));
  const int mine = lane < left ? label_of(a, (int)n0 + lane) : -1;
  const int sub = lane >> lg, c0 = lane & ((1 << lg) - 1);
  int lab[K];
#pragma unroll
  for (int k = 0; k < K; ++k) lab[k] = __shfl_sync(0xffffffffu, mine, k * per + sub);
  TR* out = rows + (n0 + sub) * a.ld_rows;
  for (int c = c0; c < vpr; c += 1 << lg) {
    Raw<VEC, TE> raw[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (lab[k] >= 0) raw[k].load(table + lab[k] * a.ld_table + c * VEC);
      else raw[k].zero();
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k * per + sub >= left) break;
      float v[VEC];
      raw[k].widen(v);
      scale_vec<VEC>(v, a.scale);
      store_vec<VEC, TR>(out + (long long)(k * per) * a.ld_rows + c * VEC, v);
    }
  }
}

template <int VEC, typename TE, typename TR>
cudaError_t launch_rows_v(const EmbedArgs& a, const TE* table, TR* rows, cudaStream_t st) {
  const int vpr = a.D / VEC;
  const int lg = vpr > 16 ? 5 : vpr > 8 ? 4 : 3, per = 32 >> lg;
  const long long N = (long long)a.B * a.U1, warps = ROWS_THREADS / 32;
  // four loads in flight per lane (eight, 19 us, or blocks of 256, 17.5, were
  // slower than 17.1 for 1024 x 101 rows of 512) once that still gives every SM
  // its warps; below, one, so that a few rows spread over the SMs
  if (N >= 64LL * num_sms() * per)
    k_embed_rows<VEC, 4>
        <<<(unsigned)cdiv(N, 4 * per * warps), ROWS_THREADS, 0, st>>>(a, lg, table, rows);
  else
    k_embed_rows<VEC, 1>
        <<<(unsigned)cdiv(N, per * warps), ROWS_THREADS, 0, st>>>(a, lg, table, rows);
  return cudaGetLastError();
}

// Widest vector (8, 2 or 1 elements) that every row of these tensors allows.
int vec_of(int D, long long ld_a, const void* pa, int size_a, long long ld_b, const void* pb,
           int size_b) {
  for (int v = 8; v > 1; v = v == 8 ? 2 : 1) {
    const int aa = v * size_a < 16 ? v * size_a : 16, ab = v * size_b < 16 ? v * size_b : 16;
    if (D % v == 0 && ld_a % v == 0 && ld_b % v == 0 && aligned_to(pa, aa) && aligned_to(pb, ab))
      return v;
  }
  return 1;
}

template <typename TE, typename TR>
cudaError_t launch_rows(const EmbedArgs& a, const void* table, void* rows, cudaStream_t st) {
  const int v = vec_of(a.D, a.ld_table, table, sizeof(TE), a.ld_rows, rows, sizeof(TR));
  if (v == 8) return launch_rows_v<8>(a, (const TE*)table, (TR*)rows, st);
  if (v == 2) return launch_rows_v<2>(a, (const TE*)table, (TR*)rows, st);
  return launch_rows_v<1>(a, (const TE*)table, (TR*)rows, st);
}

// ---- the table's gradient -----------------------------------------------------
// dE[v] = scale * sum of the dhL rows whose label is v.  The rows are listed
// by label (stably: rows of one label keep their order), so that every label
// is a run of the list, and the list is cut into chunks of equal length: the
// work does not depend on how the labels repeat.  A run inside one chunk is
// summed in registers and stored; one that crosses chunks leaves a partial row
// in each, and a second kernel adds those.  No atomics on values: the order of
// every sum follows from the labels alone.  Rows without a label carry the
// label V.

constexpr int SORT_THREADS = 1024, SORT_WARPS = SORT_THREADS / 32;

// The list of few rows, by label ranges: block c owns labels [c r, (c+1) r) and
// reads every row's label.  First it counts its own labels per warp segment and
// the rows of smaller labels, which gives every label's place; then each warp
// walks its segment in order and lists the rows.  One launch, 6.5 us for 1296
// rows and 9 for 4096 (V 16384, little to clear), where the radix sort below takes
// three, 15 us for 4097; every block reads all labels, so far beyond GROUP_MAX_ROWS
// the radix sort is the shorter (at 103,424 rows 16 us against 23).
//
// Table rows that no label names are cleared here and in the two kernels of
// the sums, a share each (ClearShare): the stores of a large table take longer
// than the rest and drain under it.
constexpr int GROUP_MAX_ROWS = 4096, GROUP_MAX_RANGE = 384;

struct ClearShare {
  int range;                // labels per group
  int j0, j1;               // this kernel's share of each group's labels
  const uint8_t* present;   // [V], NULL: nothing to clear
};

// Clear the share's rows of group g, one row per warp at a time.
__device__ __forceinline__ void clear_rows(const ClearShare& s, int g, int V, int D,
                                           float* dtable, long long ld, int v4) {
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  for (int j = s.j0 + (threadIdx.x >> 5); j < s.j1; j += warps) {
    const int v = g * s.range + j;
    if (v >= V || s.present[v]) continue;
    float* row = dtable + v * ld;
    if (v4) {
      for (int d = 4 * lane; d < D; d += 128) *(float4*)(row + d) = make_float4(0, 0, 0, 0);
    } else {
      for (int d = lane; d < D; d += 32) row[d] = 0.f;
    }
  }
}

__global__ void __launch_bounds__(SORT_THREADS)
k_embed_group(EmbedArgs a, ClearShare cs, int32_t* __restrict__ lkey, int32_t* __restrict__ lidx,
              int32_t* __restrict__ live, uint8_t* present, float* __restrict__ dtable, int v4) {
  extern __shared__ __align__(16) int32_t sm[];  // [SORT_WARPS][range] counters, [range] totals
  __shared__ __align__(16) int32_t key[GROUP_MAX_ROWS];
  __shared__ int wsum[SORT_WARPS], base_s;
  const int range = cs.range;
  int32_t* cnt = sm;
  int32_t* total = sm + SORT_WARPS * range;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int N = a.B * a.U1, NP = (N + 127) / 128 * 128;
  const int v0 = blockIdx.x * range, r = min(range, a.V - v0);
  for (int i = tid; i < SORT_WARPS * range; i += SORT_THREADS) cnt[i] = 0;
  for (int n = tid; n < NP; n += SORT_THREADS) {
    const int v = n < N ? label_of(a, n) : -1;
    key[n] = v < 0 ? a.V : v;
  }
  __syncthreads();
  // The blocks of the sums are not let in early: waiting on the SMs they take the
  // room of the clearing blocks (27.3 us against 22.7 for 1296 rows, V 16384).
  const int seg = (int)cdiv(NP / 128, SORT_WARPS) * 128;
  const int n0 = min(NP, warp * seg), n1 = min(NP, n0 + seg);
  int32_t* mycnt = cnt + warp * range;
  int below = 0;
  for (int n = n0 + 4 * lane; n < n1; n += 128) {
    const int4 q = *(const int4*)(key + n);
    const int k[4] = {q.x - v0, q.y - v0, q.z - v0, q.w - v0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      below += k[i] < 0;
      if ((unsigned)k[i] < (unsigned)r) atomicAdd(mycnt + k[i], 1);
    }
  }
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0) wsum[warp] = below;
  __syncthreads();
  // places: of a label among the smaller ones, of a warp's rows in their label
  if (warp == 0) {
    const int x = __reduce_add_sync(0xffffffffu, wsum[lane]);
    if (lane == 0) base_s = x;
  }
  for (int j = tid; j < r; j += SORT_THREADS) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < SORT_WARPS; ++w) {
      const int c = cnt[w * range + j];
      cnt[w * range + j] = run;
      run += c;
    }
    total[j] = run;
    present[v0 + j] = run != 0;
  }
  __syncthreads();
  clear_rows(cs, blockIdx.x, a.V, a.D, dtable, a.ld_table, v4);
  if (warp == 0) {
    int run = base_s;
    for (int j0 = 0; j0 < r; j0 += 32) {
      const int v = j0 + lane < r ? total[j0 + lane] : 0;
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (j0 + lane < r) total[j0 + lane] = run + x - v;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0 && v0 + r == a.V) *live = run;
  }
  __syncthreads();
  for (int n = n0; n < n1; n += 32) {
    const int k = key[n + lane] - v0;
    const bool in = (unsigned)k < (unsigned)r;
    if (!__any_sync(0xffffffffu, in)) continue;
    const unsigned peers = __match_any_sync(0xffffffffu, in ? k : -1);
    const int rank = __popc(peers & ((1u << lane) - 1));
    if (in) {
      const int pos = total[k] + mycnt[k] + rank;
      lkey[pos] = k + v0;
      lidx[pos] = n + lane;
    }
    __syncwarp();
    if (in && rank == 0) mycnt[k] += __popc(peers);
    __syncwarp();
  }
}

// The list by a radix sort, least significant digit first, for more rows or
// labels than that (rows without a label come last).  Block c owns the c-th
// range of `per` list entries.  k_embed_hist counts the first digit per
// block; every scatter pass moves its entries and counts the next digit at
// their destination (integer atomics: the counts do not depend on order).
struct SortArgs {
  int N, per, blocks;
  int shift, bits;            // this pass's digit
  int next_shift, next_bits;  // the next pass's digit (bits 0: none)
  const int32_t* key_in;
  const int32_t* idx_in;      // NULL: entry n is row n
  int32_t* key_out;
  int32_t* idx_out;
  const int32_t* hist;        // [blocks][1 << bits]
  int32_t* hist_next;
};

constexpr int MAX_DIGIT_BITS = 8;
constexpr int MAX_DIGITS = 1 << MAX_DIGIT_BITS;

// zero: counts of the later passes, cleared here
__global__ void __launch_bounds__(SORT_THREADS)
k_embed_hist(EmbedArgs a, SortArgs s, int32_t* __restrict__ key, int32_t* __restrict__ hist,
             int32_t* __restrict__ zero, int nzero) {
  __shared__ int cnt[MAX_DIGITS];
  const int R = 1 << s.bits;
  for (int d = threadIdx.x; d < R; d += SORT_THREADS) cnt[d] = 0;
  for (int i = blockIdx.x * SORT_THREADS + threadIdx.x; i < nzero; i += gridDim.x * SORT_THREADS)
    zero[i] = 0;
  __syncthreads();
  const int n1 = (int)min((long long)s.N, (long long)(blockIdx.x + 1) * s.per);
  for (int n = blockIdx.x * s.per + threadIdx.x; n < n1; n += SORT_THREADS) {
    int v = label_of(a, n);
    v = v < 0 ? a.V : v;
    key[n] = v;
    atomicAdd(&cnt[v & (R - 1)], 1);
  }
  __syncthreads();
  ptx::griddep_launch();
  for (int d = threadIdx.x; d < R; d += SORT_THREADS) hist[blockIdx.x * R + d] = cnt[d];
}

__global__ void __launch_bounds__(SORT_THREADS) k_embed_scatter(SortArgs s) {
  constexpr int WARPS = SORT_WARPS;
  __shared__ uint16_t wcnt[WARPS][MAX_DIGITS];
  __shared__ int base[MAX_DIGITS];
  __shared__ int parts[SORT_THREADS], before[SORT_THREADS];
  const int R = 1 << s.bits, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < WARPS * MAX_DIGITS / 2; i += SORT_THREADS) ((uint32_t*)wcnt)[i] = 0;
  ptx::griddep_wait();
  const int n1 = (int)min((long long)s.N, (long long)(blockIdx.x + 1) * s.per);
  // (a tile's entries are asked for ahead of what they wait for)
  int n = blockIdx.x * s.per + tid;
  int next_key = n < n1 ? s.key_in[n] : 0, next_row = n < n1 && s.idx_in ? s.idx_in[n] : n;
  // where the block's entries of digit d begin: all smaller digits, and the
  // earlier blocks' entries of the same one
  {
    const int d = tid & (R - 1), part = tid >> s.bits, np = SORT_THREADS >> s.bits;
    int all = 0, bef = 0;
#pragma unroll 4
    for (int c = part; c < s.blocks; c += np) {
      const int h = s.hist[c * R + d];
      all += h;
      if (c < (int)blockIdx.x) bef += h;
    }
    parts[tid] = all;
    before[tid] = bef;
    __syncthreads();
    if (tid < R) {
      for (int q = 1; q < np; ++q) {
        all += parts[tid + q * R];
        bef += before[tid + q * R];
      }
      base[tid] = all;
      before[tid] = bef;
    }
    __syncthreads();
    if (warp == 0) {  // exclusive scan of the digit totals
      int run = 0;
      for (int d0 = 0; d0 < R; d0 += 32) {
        const int v = d0 + lane < R ? base[d0 + lane] : 0;
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (d0 + lane < R) base[d0 + lane] = run + x - v + before[d0 + lane];
        run += __shfl_sync(0xffffffffu, x, 31);
      }
    }
  }
  ptx::griddep_launch();
  for (int t0 = blockIdx.x * s.per; t0 < n1; t0 += SORT_THREADS) {
    const bool in = n < n1;
    const int key = next_key, row = next_row;
    n += SORT_THREADS;
    if (n < n1) {
      next_key = s.key_in[n];
      next_row = s.idx_in ? s.idx_in[n] : n;
    }
    const int d = in ? (key >> s.shift) & (R - 1) : R;  // (R: no entry)
    if (t0 > (int)blockIdx.x * s.per) {
      __syncthreads();
      for (int i = tid; i < WARPS * MAX_DIGITS / 2; i += SORT_THREADS) ((uint32_t*)wcnt)[i] = 0;
    }
    __syncthreads();
    const unsigned peers = __match_any_sync(0xffffffffu, d);
    const int rank = __popc(peers & ((1u << lane) - 1));
    if (in && rank == 0) wcnt[warp][d] = (uint16_t)__popc(peers);
    __syncthreads();
    if (tid < R) {  // entries of the digit in earlier warps of the tile
      int run = 0;
#pragma unroll 8
      for (int w = 0; w < WARPS; ++w) {
        const int c = wcnt[w][tid];
        wcnt[w][tid] = (uint16_t)run;
        run += c;
      }
      parts[tid] = run;
    }
    __syncthreads();
    if (in) {
      const int pos = base[d] + wcnt[warp][d] + rank;
      s.key_out[pos] = key;
      s.idx_out[pos] = row;
      if (s.next_bits)
        atomicAdd(s.hist_next + (pos / s.per << s.next_bits) +
                      ((key >> s.next_shift) & ((1 << s.next_bits) - 1)), 1);
    }
    __syncthreads();
    if (tid < R) base[tid] += parts[tid];
  }
}

// ---- sums -----------------------------------------------------------------
// A block owns SUM_WARPS * E list entries and 32 * VEC columns; a warp sums E
// entries, FLY rows' loads in flight, and its first and last run meet the
// other warps' in shared memory (slots 2w and 2w + 1).  Bound by reading the
// rows, each once.  E = 32 amortises a warp's start; few rows take E = 8, one
// round of loads, so that more warps share them.
struct SumArgs {
  int n, V, D;
  const int32_t* live;  // list length on the device (NULL: n)
  const int32_t* key;
  const int32_t* idx;
  long long ld_src;
  float scale;
  float* dtable;
  long long ld_table;
  int chunks;           // blocks past them clear table rows that no label names
  ClearShare clear;     // (listed by label ranges; else looked up in the list)
  int v4;
  float* part;          // partial rows: chunk c's head at 2c, its tail at 2c + 1
  long long ldp;
};

constexpr int SUM_WARPS = 8;

template <int E, int VEC, typename TS>
__global__ void __launch_bounds__(SUM_WARPS * 32, 4)
k_embed_sum(SumArgs a, const TS* __restrict__ src) {
  constexpr int WARPS = SUM_WARPS;
  constexpr int FLY = VEC * sizeof(TS) > 16 ? 4 : 8;  // (four blocks an SM: 64 registers)
  __shared__ float sv[2 * WARPS][32 * VEC];
  __shared__ int skey[2 * WARPS], sused[2 * WARPS];
  struct alignas(16) Entry { long long off; int key, pad; };
  __shared__ Entry ent[WARPS][E];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = (blockIdx.y * 32 + lane) * VEC;
  const bool col_ok = col < a.D;
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int n = a.live ? *a.live : a.n;
  if ((int)blockIdx.x >= a.chunks) {
    if (blockIdx.y) return;
    if (a.clear.present) {
      clear_rows(a.clear, blockIdx.x - a.chunks, a.V, a.D, a.dtable, a.ld_table, a.v4);
      return;
    }
    // eight labels a warp, looked up in the list
    const long long v0 = ((long long)(blockIdx.x - a.chunks) * WARPS + warp) * 8;
    const long long v = v0 + lane;
    bool absent = false;
    if (lane < 8 && v < a.V) {
      int lo = 0, hi = n;  // first entry with a key >= v
      while (lo < hi) {
        const int mid = (int)(((long long)lo + hi) >> 1);
        if (a.key[mid] < v) lo = mid + 1;
        else hi = mid;
      }
      absent = lo == n || a.key[lo] != (int)v;
    }
    unsigned m = __ballot_sync(0xffffffffu, absent);
    const float z[VEC] = {};
    while (m) {
      const int r = __ffs(m) - 1;
      m &= m - 1;
      for (int d = lane * VEC; d < a.D; d += 32 * VEC)
        store_vec<VEC, float>(a.dtable + (v0 + r) * a.ld_table + d, z);
    }
    return;
  }
  auto store_row = [&](int v, float (&acc)[VEC]) {
    if (!col_ok) return;
    float o[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = acc[i];
    scale_vec<VEC>(o, a.scale);
    store_vec<VEC, float>(a.dtable + v * a.ld_table + col, o);
  };
  const long long b0 = (long long)blockIdx.x * WARPS * E, b1 = b0 + WARPS * E;
  if (b0 >= n) return;
  const long long e0 = b0 + warp * E;
  const int here = (int)max(0LL, min((long long)E, n - e0));
  const int mykey = lane < here ? a.key[e0 + lane] : a.V;
  const long long myrow = lane < here ? a.idx[e0 + lane] : 0;
  const int prev = here > 0 && e0 > 0 ? a.key[e0 - 1] : -1;
  const int next = e0 + E < n ? a.key[e0 + E] : -1;
  const int bprev = b0 > 0 ? a.key[b0 - 1] : -1;
  const int bnext = b1 < n ? a.key[b1] : -1;
  // rows without a label (V) are last: they are no entries
  const int cnt = __popc(__ballot_sync(0xffffffffu, mykey != a.V));
  if (lane < E) ent[warp][lane] = Entry{myrow * a.ld_src, mykey, 0};
  if (lane < 2) {
    skey[2 * warp + lane] = a.V;
    sused[2 * warp + lane] = 0;
  }
  __syncwarp();
  float acc[VEC] = {};
  int cur = __shfl_sync(0xffffffffu, mykey, 0);
  bool first = true;  // the run that holds the segment's first entry
  auto flush = [&](bool last) {
    if (cur == a.V) return;
    const bool left = first && prev == cur, right = last && next == cur;
    if (!left && !right) {
      store_row(cur, acc);
      return;
    }
    const int slot = 2 * warp + !left;
#pragma unroll
    for (int i = 0; i < VEC; ++i) sv[slot][i * 32 + lane] = acc[i];
    if (lane == 0) {
      skey[slot] = cur;
      sused[slot] = 1;
      // (a run through the whole segment: the empty tail keeps its key, so
      // that the pieces stay neighbours)
      if (left && right) skey[slot + 1] = cur;
    }
  };
  const TS* mycol = src + (col_ok ? col : 0);
#pragma unroll 1
  for (int j0 = 0; j0 < cnt; j0 += FLY) {
    Raw<VEC, TS> raw[FLY];
    int key[FLY];
#pragma unroll
    for (int j = 0; j < FLY; ++j) {
      // (past the last entry: the last one again, not added)
      const Entry e = ent[warp][min(j0 + j, cnt - 1)];
      key[j] = e.key;
      raw[j].load(mycol + e.off);
    }
#pragma unroll
    for (int j = 0; j < FLY; ++j) {
      if (j0 + j >= cnt) break;
      if (key[j] != cur) {
        flush(false);
        cur = key[j];
        first = false;
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
      }
      float x[VEC];
      raw[j].widen(x);
      add_vec<VEC>(acc, x);
    }
  }
  flush(true);
  __syncthreads();
  if (warp != 0) return;
  // the warps' pieces, in order
  const int slotkey = lane < 2 * WARPS ? skey[lane] : a.V;
  if (!__any_sync(0xffffffffu, slotkey != a.V)) return;
  const int slotused = lane < 2 * WARPS ? sused[lane] : 0;
  cur = __shfl_sync(0xffffffffu, slotkey, 0);
  first = true;
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  auto flush_block = [&](bool last) {
    if (cur == a.V) return;
    const bool left = first && bprev == cur, right = last && bnext == cur;
    if (!left && !right) store_row(cur, acc);
    else if (col_ok) store_vec<VEC, float>(a.part + (2LL * blockIdx.x + !left) * a.ldp + col, acc);
  };
#pragma unroll
  for (int s = 0; s < 2 * WARPS; ++s) {
    const int k = __shfl_sync(0xffffffffu, slotkey, s);
    if (k != cur) {
      flush_block(false);
      cur = k;
      first = false;
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
    }
    if (__shfl_sync(0xffffffffu, slotused, s)) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += sv[s][i * 32 + lane];
    }
  }
  flush_block(true);
}

// Runs that cross chunks: the block of the chunk in which such a run begins
// finds the chunk in which it ends and adds its pieces, a contiguous share per
// warp, then the warps' sums in order.
template <int E, int VEC>
__global__ void __launch_bounds__(SUM_WARPS * 32) k_embed_join(SumArgs a) {
  constexpr int CHUNK = SUM_WARPS * E;
  __shared__ float sv[SUM_WARPS][32 * VEC];
  __shared__ int end_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = (blockIdx.y * 32 + lane) * VEC;
  const int c = blockIdx.x;
  ptx::griddep_wait();
  if (c >= a.chunks - 1) {
    if (blockIdx.y == 0)
      clear_rows(a.clear, c - max(0, a.chunks - 1), a.V, a.D, a.dtable, a.ld_table, a.v4);
    return;
  }
  const int n = a.live ? *a.live : a.n;
  const long long e0 = (long long)c * CHUNK, e1 = e0 + CHUNK;
  if (e1 >= n) return;
  const int k = a.key[e1 - 1];
  if (k == a.V || a.key[e1] != k) return;
  if (e0 > 0 && a.key[e0 - 1] == k) return;  // it began earlier
  // last chunk of the run: the first after c whose next entry is another label
  if (threadIdx.x == 0) end_s = 0x7fffffff;
  __syncthreads();
  int last = 0;
  for (int d = c + 1;; d += SUM_WARPS * 32) {
    const long long e = ((long long)d + threadIdx.x + 1) * CHUNK;
    if (e >= n || a.key[e] != k) atomicMin(&end_s, d + threadIdx.x);
    __syncthreads();
    last = end_s;
    __syncthreads();
    if (last != 0x7fffffff) break;
  }
  const int pieces = last - c + 1, share = (pieces + SUM_WARPS - 1) / SUM_WARPS;
  const int p0 = warp * share, p1 = min(pieces, p0 + share);
  float acc[VEC] = {};
  if (col < a.D) {
#pragma unroll 4
    for (int p = p0; p < p1; ++p) {  // piece 0 is chunk c's tail, the others are heads
      Raw<VEC, float> raw;
      raw.load_late(a.part + (2LL * (c + p) + (p == 0)) * a.ldp + col);
      float x[VEC];
      raw.widen(x);
      add_vec<VEC>(acc, x);
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) sv[warp][i * 32 + lane] = acc[i];
  __syncthreads();
  if (warp != 0 || col >= a.D) return;
  const int busy = (pieces + share - 1) / share;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    float s = acc[i];
    for (int w = 1; w < busy; ++w) s += sv[w][i * 32 + lane];
    acc[i] = a.scale * s;
  }
  store_vec<VEC, float>(a.dtable + k * a.ld_table + col, acc);
}

bool embed_args(const rnnt_embed_dims* d, EmbedArgs* a) {
  if (!d || d->B < 0 || d->U1 < 1 || d->V < 1 || d->D < 1) return false;
  // (the sums take their columns in at most 65535 blocks of 32)
  if ((long long)d->B * d->U1 > (1LL << 30) || d->D > (1 << 20)) return false;
  if (d->sos && (d->blank < 0 || d->blank >= d->V)) return false;
  if (!op_dtype(d->table_dtype) || !op_dtype(d->row_dtype) || !isfinite(d->scale)) return false;
  if ((d->ld_table && d->ld_table < d->D) || (d->ld_rows && d->ld_rows < d->D)) return false;
  a->B = d->B; a->U1 = d->U1; a->V = d->V; a->D = d->D;
  a->blank = d->blank; a->sos = d->sos != 0; a->scale = d->scale;
  a->ld_table = d->ld_table ? d->ld_table : d->D;
  a->ld_rows = d->ld_rows ? d->ld_rows : d->D;
  return true;
}

// Workspace and launches of a gradient call.
struct EmbedPlan {
  int N;
  int range, groups;                 // listed by label ranges (groups 0: by the radix sort)
  int blocks, per, passes, bits;
  int entries;                       // list entries per warp of the sums
  int chunks;
  int ldp;
  size_t w_key[2], w_idx[2], w_live, w_present, w_hist, hist_each, w_part, total;
};

EmbedPlan embed_plan(const EmbedArgs& a) {
  EmbedPlan p{};
  p.N = a.B * a.U1;
  size_t o = 0;
  auto put = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes); return at; };
  for (int i = 0; i < 2; ++i) {
    p.w_key[i] = put(4 * (size_t)p.N);
    p.w_idx[i] = put(4 * (size_t)p.N);
  }
  p.w_live = put(4);
  // (152: the SMs; the layout may not depend on the device that runs it)
  p.range = (int)cdiv(a.V, 152);
  if (p.N > 0 && p.N <= GROUP_MAX_ROWS && p.range <= GROUP_MAX_RANGE) {
    p.groups = (int)cdiv(a.V, p.range);
    p.w_present = put((size_t)a.V);
  } else {
    int bits = 1;
    while ((1LL << bits) <= a.V) ++bits;  // labels 0 to V
    p.passes = (int)cdiv(bits, MAX_DIGIT_BITS);
    p.bits = (int)cdiv(bits, p.passes);
    // at most one block per SM, whole tiles of SORT_THREADS entries each (every
    // block reads all blocks' counts, so more blocks would read more)
    const long long tiles = cdiv(p.N, SORT_THREADS);
    p.per = (int)cdiv(tiles, tiles < 152 ? (tiles ? tiles : 1) : 152) * SORT_THREADS;
    p.blocks = p.N ? (int)cdiv(p.N, p.per) : 0;
    p.hist_each = (size_t)p.blocks << p.bits;
    p.w_hist = put(4 * p.hist_each * p.passes);
  }
  // one round of loads a warp until that fills the SMs' warps several times
  p.entries = p.N <= 16384 ? 8 : 32;
  p.chunks = (int)cdiv(p.N, SUM_WARPS * p.entries);
  p.ldp = (int)cdiv(a.D, 8) * 8;
  p.w_part = put(8 * (size_t)p.chunks * p.ldp);
  p.total = o;
  return p;
}

// A launch that may start its set-up under the previous kernel's tail (the
// kernels wait with griddep_wait before they read).
template <typename... KA, typename... A>
cudaError_t launch_dep(void (*k)(KA...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                       A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

cudaError_t launch_group(const EmbedArgs& a, const EmbedPlan& p, const ClearShare& cs,
                         int32_t* lkey, int32_t* lidx, int32_t* live, float* dtable, int v4,
                         cudaStream_t st) {
  const size_t smem = 4 * (size_t)(SORT_WARPS + 1) * p.range;
  static std::atomic<bool> opted_in[kDeviceSlots];
  std::atomic<bool>& opted = opted_in[device_slot()];
  if (!opted.load()) {
    const cudaError_t e = cudaFuncSetAttribute(k_embed_group,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               4 * (SORT_WARPS + 1) * GROUP_MAX_RANGE);
    if (e != cudaSuccess) return e;
    opted.store(true);
  }
  k_embed_group<<<p.groups, SORT_THREADS, smem, st>>>(a, cs, lkey, lidx, live,
                                                      (uint8_t*)cs.present, dtable, v4);
  return cudaGetLastError();
}

template <int E, int VEC, typename TS>
cudaError_t launch_sums_v(SumArgs s, const void* src, int clear, ClearShare last,
                          cudaStream_t st) {
  const unsigned cols = (unsigned)cdiv(s.D, 32 * VEC);
  const cudaError_t e = launch_dep(k_embed_sum<E, VEC, TS>, dim3(s.chunks + clear, cols),
                                   SUM_WARPS * 32, 0, st, s, (const TS*)src);
  if (e != cudaSuccess) return e;
  s.clear = last;
  const int join = (s.chunks > 1 ? s.chunks - 1 : 0) + (last.present ? clear : 0);
  if (!join) return cudaSuccess;
  return launch_dep(k_embed_join<E, VEC>, dim3(join, cols), SUM_WARPS * 32, 0, st, s);
}

template <typename TS>
cudaError_t launch_sums(const SumArgs& s, const void* src, int clear, const ClearShare& last,
                        int entries, int vec, cudaStream_t st) {
  if (entries == 8) {
    if (vec == 8) return launch_sums_v<8, 8, TS>(s, src, clear, last, st);
    if (vec == 2) return launch_sums_v<8, 2, TS>(s, src, clear, last, st);
    return launch_sums_v<8, 1, TS>(s, src, clear, last, st);
  }
  if (vec == 8) return launch_sums_v<32, 8, TS>(s, src, clear, last, st);
  if (vec == 2) return launch_sums_v<32, 2, TS>(s, src, clear, last, st);
  return launch_sums_v<32, 1, TS>(s, src, clear, last, st);
}

}  // namespace
}  // namespace rnnt

using namespace rnnt;

extern "C" {

rnnt_status rnnt_ops_status(const int32_t* status, rnnt_stream stream, int32_t* word) {
  if (!status) return RNNT_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  int32_t w = 0;
  OPS_CHECK(cudaMemcpyAsync(&w, status, sizeof(int32_t), cudaMemcpyDeviceToHost, st));
  OPS_CHECK(cudaStreamSynchronize(st));
  if (word) *word = w;
  const rnnt_status order[] = {RNNT_ERR_LENGTH_RANGE, RNNT_ERR_LABEL_RANGE, RNNT_ERR_TIMEOUT};
  for (rnnt_status c : order)
    if (w & status_bit(c)) return c;
  return RNNT_OK;
}

size_t rnnt_embed_workspace_bytes(const rnnt_embed_dims* dims) {
  EmbedArgs a;
  return embed_args(dims, &a) ? embed_plan(a).total : 0;
}

rnnt_status rnnt_embed_fwd(const rnnt_embed_dims* dims, const int32_t* ids, const int32_t* U_len,
                           const void* table, void* rows, int32_t* status, rnnt_stream stream) {
  EmbedArgs a;
  if (!embed_args(dims, &a)) return RNNT_ERR_INVALID_ARG;
  if (a.B == 0) return RNNT_OK;
  if (!ids || !table || !rows) return RNNT_ERR_INVALID_ARG;
  if (!aligned_to(ids, 4) || !aligned_to(table, op_size(dims->table_dtype)) ||
      !aligned_to(rows, op_size(dims->row_dtype)) || !aligned_to(U_len, 4) ||
      !aligned_to(status, 4))
    return RNNT_ERR_INVALID_ARG;
  a.ids = ids; a.U_len = U_len; a.status = status;
  cudaStream_t st = (cudaStream_t)stream;
  using bf = __nv_bfloat16;
  ProfScope ps("embed_rows", st);
  const bool rf = dims->row_dtype == RNNT_F32;
  if (dims->table_dtype == RNNT_F32)
    OPS_CHECK((rf ? launch_rows<float, float>(a, table, rows, st)
                  : launch_rows<float, bf>(a, table, rows, st)));
  else
    OPS_CHECK((rf ? launch_rows<bf, float>(a, table, rows, st)
                  : launch_rows<bf, bf>(a, table, rows, st)));
  return RNNT_OK;
}

rnnt_status rnnt_embed_bwd(const rnnt_embed_dims* dims, const int32_t* ids, const int32_t* U_len,
                           const void* drows, float* dtable, void* ws, size_t ws_bytes,
                           int32_t* status, rnnt_stream stream) {
  EmbedArgs a;
  if (!embed_args(dims, &a)) return RNNT_ERR_INVALID_ARG;
  if (!dtable || !ws || (a.B > 0 && (!ids || !drows))) return RNNT_ERR_INVALID_ARG;
  if (!aligned_to(ids, 4) || !aligned_to(drows, op_size(dims->row_dtype)) ||
      !aligned_to(dtable, 4) || !aligned_to(U_len, 4) || !aligned_to(status, 4) ||
      !aligned_to(ws, ALIGN))
    return RNNT_ERR_INVALID_ARG;
  if (ws_bytes < rnnt_embed_workspace_bytes(dims)) return RNNT_ERR_WORKSPACE_TOO_SMALL;
  a.ids = ids; a.U_len = U_len; a.status = status;
  cudaStream_t st = (cudaStream_t)stream;
  const EmbedPlan p = embed_plan(a);
  char* w = (char*)ws;
  auto at = [&](size_t off) { return (int32_t*)(w + off); };
  int out = 0;  // which of the two list buffers holds the list
  const int v4 = a.D % 4 == 0 && a.ld_table % 4 == 0 && aligned_to(dtable, 16);
  ClearShare cs{};
  if (p.groups) {
    cs.range = p.range;
    cs.j1 = p.range * 3 / 8;
    cs.present = (const uint8_t*)(w + p.w_present);
    OPS_LAUNCH("embed_list", launch_group(a, p, cs, at(p.w_key[0]), at(p.w_idx[0]), at(p.w_live),
                                          dtable, v4, st));
  } else if (p.N > 0) {
    ProfScope ps("embed_list", st);
    ps.set_kernels(1 + p.passes);
    SortArgs s{};
    s.N = p.N; s.per = p.per; s.blocks = p.blocks; s.bits = p.bits;
    int32_t* hist = at(p.w_hist);
    k_embed_hist<<<p.blocks, SORT_THREADS, 0, st>>>(a, s, at(p.w_key[1]), hist,
                                                    hist + p.hist_each,
                                                    (int)(p.hist_each * (p.passes - 1)));
    OPS_CHECK(cudaGetLastError());
    for (int k = 0; k < p.passes; ++k) {
      out = k & 1;
      s.key_in = at(p.w_key[1 - out]);
      s.idx_in = k ? at(p.w_idx[1 - out]) : nullptr;
      s.key_out = at(p.w_key[out]);
      s.idx_out = at(p.w_idx[out]);
      s.shift = k * p.bits;
      s.next_shift = s.shift + p.bits;
      s.next_bits = k + 1 < p.passes ? p.bits : 0;
      s.hist = hist + k * p.hist_each;
      s.hist_next = hist + (k + 1) * p.hist_each;
      OPS_CHECK(launch_dep(k_embed_scatter, dim3(p.blocks), SORT_THREADS, 0, st, s));
    }
  }
  ProfScope ps("embed_grad", st);
  ps.set_kernels(p.chunks < 2 && !p.groups ? 1 : 2);
  SumArgs s{};
  s.n = p.N; s.V = a.V; s.D = a.D;
  s.live = p.groups ? at(p.w_live) : nullptr;
  s.key = at(p.w_key[out]);
  s.idx = at(p.w_idx[out]);
  s.ld_src = a.ld_rows;
  s.scale = a.scale;
  s.dtable = dtable; s.ld_table = a.ld_table;
  s.chunks = p.chunks;
  s.part = (float*)(w + p.w_part);
  s.ldp = p.ldp;
  s.v4 = v4;
  ClearShare last{};
  int clear = (int)cdiv(a.V, 8 * SUM_WARPS);
  if (p.groups) {
    clear = p.groups;
    last = s.clear = cs;
    s.clear.j0 = cs.j1;
    s.clear.j1 = last.j0 = p.range * 3 / 4;
    last.j1 = p.range;
  }
  const int vec = vec_of(a.D, a.ld_table, dtable, 4, a.ld_rows, drows, op_size(dims->row_dtype));
  OPS_CHECK(dims->row_dtype == RNNT_F32
                ? launch_sums<float>(s, drows, clear, last, p.entries, vec, st)
                : launch_sums<__nv_bfloat16>(s, drows, clear, last, p.entries, vec, st));
  return RNNT_OK;
}

}  // extern "C"
