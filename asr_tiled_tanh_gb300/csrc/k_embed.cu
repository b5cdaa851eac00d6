// k_embed.cu -- the prediction network's label embedding (include/rnnt_ops.h).
#include <algorithm>

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
// table's rows come from L2): a block holds as many rows as fit its threads, a
// thread owns VEC consecutive columns of K rows, whose loads are in flight
// together.  VEC = 8 needs 16-byte aligned rows; others take one column.
template <int VEC, typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = to_f<T>(*p);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 q = __ldg((const float4*)(p + i));
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
  } else if constexpr (VEC == 4) {
    const uint2 q = __ldg((const uint2*)p);
    v[0] = ptx::bf16lo(q.x); v[1] = ptx::bf16hi(q.x);
    v[2] = ptx::bf16lo(q.y); v[3] = ptx::bf16hi(q.y);
  } else {
    const uint4 q = __ldg((const uint4*)p);
    v[0] = ptx::bf16lo(q.x); v[1] = ptx::bf16hi(q.x);
    v[2] = ptx::bf16lo(q.y); v[3] = ptx::bf16hi(q.y);
    v[4] = ptx::bf16lo(q.z); v[5] = ptx::bf16hi(q.z);
    v[6] = ptx::bf16lo(q.w); v[7] = ptx::bf16hi(q.w);
  }
}
template <int VEC, typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    *p = from_f<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4)
      *(float4*)(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    static_assert(VEC == 8, "bf16 stores are 16 bytes");
    *(uint4*)p = make_uint4(ptx::pack_bf16x2(v[0], v[1]), ptx::pack_bf16x2(v[2], v[3]),
                            ptx::pack_bf16x2(v[4], v[5]), ptx::pack_bf16x2(v[6], v[7]));
  }
}

constexpr int ROWS_THREADS = 256;

template <int VEC, int K, typename TE, typename TR>
__global__ void __launch_bounds__(ROWS_THREADS)
k_embed_rows(EmbedArgs a, const TE* __restrict__ table, TR* __restrict__ rows) {
  const int vpr = a.D / VEC;                     // vectors per row
  const int tpr = min(vpr, ROWS_THREADS);        // threads per row
  const int rpb = ROWS_THREADS / tpr;            // rows per pass of the block
  const int r = threadIdx.x / tpr, c0 = threadIdx.x - r * tpr;
  if (r >= rpb) return;
  const int N = a.B * a.U1;
  const long long n0 = (long long)blockIdx.x * rpb * K + r;
  int lab[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const long long n = n0 + (long long)k * rpb;
    lab[k] = n < N ? label_of(a, (int)n) : -1;
  }
  for (int c = c0; c < vpr; c += tpr) {
    float v[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (lab[k] >= 0) {
        load_vec<VEC, TE>(table + lab[k] * a.ld_table + c * VEC, v[k]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[k][i] = 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const long long n = n0 + (long long)k * rpb;
      if (n < N) {
        if (lab[k] >= 0) {  // (0 exactly where there is no label, whatever the scale)
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[k][i] *= a.scale;
        }
        store_vec<VEC, TR>(rows + n * a.ld_rows + c * VEC, v[k]);
      }
    }
  }
}

template <int VEC, typename TE, typename TR>
cudaError_t launch_rows_v(const EmbedArgs& a, const TE* table, TR* rows, cudaStream_t st) {
  const int vpr = a.D / VEC, rpb = ROWS_THREADS / std::min(vpr, ROWS_THREADS);
  const long long N = (long long)a.B * a.U1;
  // four rows a thread once every SM has several blocks of them; below, one,
  // so that a few rows still spread over the SMs
  if (N >= 32LL * num_sms() * rpb)
    k_embed_rows<VEC, 4><<<(unsigned)cdiv(N, 4 * rpb), ROWS_THREADS, 0, st>>>(a, table, rows);
  else
    k_embed_rows<VEC, 1><<<(unsigned)cdiv(N, rpb), ROWS_THREADS, 0, st>>>(a, table, rows);
  return cudaGetLastError();
}

template <typename TE, typename TR>
cudaError_t launch_rows(const EmbedArgs& a, const void* table, void* rows, cudaStream_t st) {
  const bool v8 = a.D % 8 == 0 && a.ld_table % 8 == 0 && a.ld_rows % 8 == 0 &&
                  aligned_to(table, 16) && aligned_to(rows, 16);
  return v8 ? launch_rows_v<8>(a, (const TE*)table, (TR*)rows, st)
            : launch_rows_v<1>(a, (const TE*)table, (TR*)rows, st);
}

// ---- the table's gradient -----------------------------------------------------
// dE[v] = scale * sum of the dhL rows whose label is v.  The rows' labels are
// sorted (stably: rows of one label keep their order), so that every label is
// a run of the sorted list, and the list is cut into chunks of equal length:
// the work does not depend on how the labels repeat.  A run inside one chunk
// is summed in registers and stored; a run that crosses chunks leaves one
// partial row in each, and the partial rows form the next level's (much
// shorter) sorted list.  No atomics on values: the order of every sum follows
// from the labels alone.  Rows without a label carry the label V and sort last.

// Stable sort of few rows by counting: a warp finds row i's place as the number
// of rows with a smaller label plus the earlier ones with the same label.  N^2
// comparisons, but one launch; at 4096 rows as long as the radix passes.
constexpr int RANK_MAX = 4096;
constexpr int SORT_THREADS = 1024;

__global__ void __launch_bounds__(SORT_THREADS)
k_embed_rank(EmbedArgs a, int32_t* __restrict__ skey, int32_t* __restrict__ sidx) {
  __shared__ __align__(16) int32_t key[RANK_MAX];
  const int N = a.B * a.U1, N4 = (N + 127) / 128 * 128;
  for (int n = threadIdx.x; n < N4; n += SORT_THREADS) {
    const int v = n < N ? label_of(a, n) : a.V;
    key[n] = v < 0 ? a.V : v;
  }
  __syncthreads();
  ptx::griddep_launch();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * (SORT_THREADS / 32) + (threadIdx.x >> 5);
  if (i >= N) return;
  const int k = key[i];
  int below = 0;
  for (int j = 4 * lane; j < N4; j += 128) {
    const int4 q = *(const int4*)(key + j);
    below += q.x < k + (j < i);
    below += q.y < k + (j + 1 < i);
    below += q.z < k + (j + 2 < i);
    below += q.w < k + (j + 3 < i);
  }
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0) {
    skey[below] = k;
    sidx[below] = i;
  }
}

// Radix sort, least significant digit first, for more rows.  Block c owns the
// c-th range of `per` list entries.  k_embed_hist counts the first digit per
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
  constexpr int WARPS = SORT_THREADS / 32;
  __shared__ uint16_t wcnt[WARPS][MAX_DIGITS];
  __shared__ int base[MAX_DIGITS];
  __shared__ int parts[SORT_THREADS], before[SORT_THREADS];
  const int R = 1 << s.bits, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ptx::griddep_wait();
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
  const int n1 = (int)min((long long)s.N, (long long)(blockIdx.x + 1) * s.per);
  for (int t0 = blockIdx.x * s.per; t0 < n1; t0 += SORT_THREADS) {
    const int n = t0 + tid;
    const bool in = n < n1;
    const int key = in ? s.key_in[n] : 0;
    const int row = in ? (s.idx_in ? s.idx_in[n] : n) : 0;
    const int d = in ? (key >> s.shift) & (R - 1) : R;  // (R: no entry)
    __syncthreads();
    for (int i = tid; i < WARPS * R; i += SORT_THREADS) wcnt[i >> s.bits][i & (R - 1)] = 0;
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

// One level of the sums.  A block owns WARPS * 32 list entries and 32 * VEC
// columns; a warp sums 32 entries, eight rows' loads in flight, and its first
// and last run meet the other warps' in shared memory (slots 2w and 2w + 1).
// Bound by reading the rows: each is read once, 512 bytes of it per warp.
struct SumArgs {
  int n, V, D;
  const int32_t* key;
  const int32_t* idx;   // row of src, -1: nothing to add (its key still counts)
  long long ld_src;
  float scale;
  float* dtable;
  long long ld_table;
  int chunks;           // blocks past them store zeros into labels that do not occur
  int32_t* pkey;        // next level's list (2 per chunk); unused at the last level
  int32_t* pidx;
  float* part;
  long long ldp;
};

// Sum of a run, as it leaves a warp or block: alone (its label is complete), or
// one piece of a run that continues to the left (head slot) or right only (tail).
enum { RUN_WHOLE, RUN_HEAD, RUN_TAIL };
__device__ __forceinline__ int run_kind(bool left, bool right) {
  return left ? RUN_HEAD : right ? RUN_TAIL : RUN_WHOLE;
}

template <int WARPS, int VEC, typename TS>
__global__ void __launch_bounds__(WARPS * 32)
k_embed_sum(SumArgs a, const TS* __restrict__ src) {
  __shared__ float sv[2 * WARPS][32 * VEC];
  __shared__ int skey[2 * WARPS], sused[2 * WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = (blockIdx.y * 32 + lane) * VEC;
  const bool col_ok = col < a.D;
  ptx::griddep_wait();
  ptx::griddep_launch();
  if ((int)blockIdx.x >= a.chunks) {
    // labels that do not occur: eight a warp, looked up in the sorted list
    const long long v0 = ((long long)(blockIdx.x - a.chunks) * WARPS + warp) * 8;
    const long long v = v0 + lane;
    bool absent = false;
    if (lane < 8 && v < a.V) {
      int lo = 0, hi = a.n;  // first entry with a key >= v
      while (lo < hi) {
        const int mid = (int)(((long long)lo + hi) >> 1);
        if (a.key[mid] < v) lo = mid + 1;
        else hi = mid;
      }
      absent = lo == a.n || a.key[lo] != (int)v;
    }
    unsigned m = __ballot_sync(0xffffffffu, absent);
    const float z[VEC] = {};
    while (m) {
      const int r = __ffs(m) - 1;
      m &= m - 1;
      if (col_ok) store_vec<VEC, float>(a.dtable + (v0 + r) * a.ld_table + col, z);
    }
    return;
  }
  auto store_row = [&](int v, float (&acc)[VEC]) {
    if (!col_ok) return;
    float o[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = a.scale * acc[i];
    store_vec<VEC, float>(a.dtable + v * a.ld_table + col, o);
  };
  const long long e0 = ((long long)blockIdx.x * WARPS + warp) * 32;
  const int cnt = (int)max(0LL, min(32LL, a.n - e0));
  const int mykey = lane < cnt ? a.key[e0 + lane] : a.V;
  const int myidx = lane < cnt ? a.idx[e0 + lane] : -1;
  const int prev = cnt > 0 && e0 > 0 ? a.key[e0 - 1] : -1;
  const int next = e0 + 32 < a.n ? a.key[e0 + 32] : -1;
  if (lane < 2) {
    skey[2 * warp + lane] = a.V;
    sused[2 * warp + lane] = 0;
  }
  __syncwarp();
  float acc[VEC] = {};
  int cur = __shfl_sync(0xffffffffu, mykey, 0);
  bool first = true;  // the run that holds entry 0
  auto flush = [&](bool last) {
    if (cur == a.V) return;
    const bool left = first && prev == cur, right = last && next == cur;
    const int kind = run_kind(left, right);
    if (kind == RUN_WHOLE) {
      store_row(cur, acc);
      return;
    }
    const int slot = 2 * warp + (kind == RUN_TAIL);
#pragma unroll
    for (int i = 0; i < VEC; ++i) sv[slot][lane * VEC + i] = acc[i];
    if (lane == 0) {
      skey[slot] = cur;
      sused[slot] = 1;
      // (a run through the whole segment: the empty tail keeps its key, so
      // that the pieces stay neighbours)
      if (left && right) skey[slot + 1] = cur;
    }
  };
#pragma unroll 1
  for (int j0 = 0; j0 < cnt; j0 += 8) {
    float x[8][VEC];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = __shfl_sync(0xffffffffu, mykey, j0 + j);
      const int r = __shfl_sync(0xffffffffu, myidx, j0 + j);
      if (k != a.V && r >= 0 && col_ok) {
        load_vec<VEC, TS>(src + r * a.ld_src + col, x[j]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[j][i] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = __shfl_sync(0xffffffffu, mykey, j0 + j);
      if (k != cur) {
        flush(false);
        cur = k;
        first = false;
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = x[j][i];
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] += x[j][i];
      }
    }
  }
  flush(true);
  __syncthreads();
  if (warp != 0) return;
  // the warps' pieces, in order
  const long long b0 = (long long)blockIdx.x * WARPS * 32;
  const int bprev = b0 > 0 ? a.key[b0 - 1] : -1;
  const int bnext = b0 + WARPS * 32 < a.n ? a.key[b0 + WARPS * 32] : -1;
  int hk[2] = {a.V, a.V}, hu[2] = {-1, -1};
  cur = skey[0];
  first = true;
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  auto flush_block = [&](bool last) {
    if (cur == a.V) return;
    const bool left = first && bprev == cur, right = last && bnext == cur;
    const int kind = run_kind(left, right);
    if (kind == RUN_WHOLE) {
      store_row(cur, acc);
      return;
    }
    const int t = kind == RUN_TAIL;
    const int slot = 2 * blockIdx.x + t;
    if (col_ok) store_vec<VEC, float>(a.part + slot * a.ldp + col, acc);
    hk[t] = cur;
    hu[t] = slot;
    if (left && right) hk[1] = cur;
  };
  for (int s = 0; s < 2 * WARPS; ++s) {
    const int k = skey[s];
    if (k != cur) {
      flush_block(false);
      cur = k;
      first = false;
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
    }
    if (sused[s]) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += sv[s][lane * VEC + i];
    }
  }
  flush_block(true);
  if (a.pkey && blockIdx.y == 0 && lane < 2) {
    a.pkey[2 * blockIdx.x + lane] = lane ? hk[1] : hk[0];
    a.pidx[2 * blockIdx.x + lane] = lane ? hu[1] : hu[0];
  }
}

bool embed_args(const rnnt_embed_dims* d, EmbedArgs* a) {
  if (!d || d->B < 0 || d->U1 < 1 || d->V < 1 || d->D < 1) return false;
  if ((long long)d->B * d->U1 > (1LL << 30)) return false;
  if (d->sos && (d->blank < 0 || d->blank >= d->V)) return false;
  if (!op_dtype(d->table_dtype) || !op_dtype(d->row_dtype)) return false;
  if ((d->ld_table && d->ld_table < d->D) || (d->ld_rows && d->ld_rows < d->D)) return false;
  a->B = d->B; a->U1 = d->U1; a->V = d->V; a->D = d->D;
  a->blank = d->blank; a->sos = d->sos != 0; a->scale = d->scale;
  a->ld_table = d->ld_table ? d->ld_table : d->D;
  a->ld_rows = d->ld_rows ? d->ld_rows : d->D;
  return true;
}

// Workspace and levels of a gradient call.
struct EmbedPlan {
  int N, blocks, per, passes, bits;  // blocks 0: sorted by counting
  int levels;
  long long n[8], chunks[8];         // list length and chunks of every level
  int ldp;
  size_t w_key[2], w_idx[2], w_hist, hist_each, w_pkey[8], w_pidx[8], w_part[8], total;
};

constexpr int SUM_WARPS0 = 8, SUM_WARPS1 = 32;

EmbedPlan embed_plan(const EmbedArgs& a) {
  EmbedPlan p{};
  p.N = a.B * a.U1;
  size_t o = 0;
  auto put = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes); return at; };
  for (int i = 0; i < 2; ++i) {
    p.w_key[i] = put(4 * (size_t)p.N);
    p.w_idx[i] = put(4 * (size_t)p.N);
  }
  if (p.N > RANK_MAX) {
    int bits = 1;
    while ((1LL << bits) <= a.V) ++bits;  // labels 0 to V
    p.passes = (int)cdiv(bits, MAX_DIGIT_BITS);
    p.bits = (int)cdiv(bits, p.passes);
    // at most one block per SM, whole tiles of SORT_THREADS entries each (every
    // block reads all blocks' counts, so more blocks would read more)
    const long long tiles = cdiv(p.N, SORT_THREADS);
    p.per = (int)cdiv(tiles, std::min<long long>(tiles, 152)) * SORT_THREADS;
    p.blocks = (int)cdiv(p.N, p.per);
    p.hist_each = (size_t)p.blocks << p.bits;
    p.w_hist = put(4 * p.hist_each * p.passes);
  }
  p.ldp = (int)cdiv(a.D, 4) * 4;
  long long n = p.N;
  for (int l = 0;; ++l) {
    p.n[l] = n;
    p.chunks[l] = cdiv(n, 32 * (l ? SUM_WARPS1 : SUM_WARPS0));
    p.levels = l + 1;
    if (p.chunks[l] <= 1) break;
    const size_t slots = 2 * (size_t)p.chunks[l];
    p.w_pkey[l] = put(4 * slots);
    p.w_pidx[l] = put(4 * slots);
    p.w_part[l] = put(4 * slots * p.ldp);
    n = (long long)slots;
  }
  p.total = o ? o : ALIGN;
  return p;
}

// A launch that may start its set-up under the previous kernel's tail (the
// kernels wait with griddep_wait before they read).
template <typename... KA, typename... A>
cudaError_t launch_dep(void (*k)(KA...), dim3 grid, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

template <int WARPS, typename TS>
cudaError_t launch_sum(const SumArgs& s, const void* src, unsigned blocks, bool v4,
                       cudaStream_t st) {
  const dim3 grid(blocks, (unsigned)cdiv(s.D, v4 ? 128 : 32));
  return v4 ? launch_dep(k_embed_sum<WARPS, 4, TS>, grid, WARPS * 32, st, s, (const TS*)src)
            : launch_dep(k_embed_sum<WARPS, 1, TS>, grid, WARPS * 32, st, s, (const TS*)src);
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
  int out = 0;  // which of the two list buffers holds the sorted list
  if (p.N > 0 && !p.blocks) {
    ProfScope ps("embed_sort", st);
    k_embed_rank<<<(unsigned)cdiv(p.N, SORT_THREADS / 32), SORT_THREADS, 0, st>>>(
        a, at(p.w_key[0]), at(p.w_idx[0]));
    OPS_CHECK(cudaGetLastError());
  } else if (p.N > 0) {
    ProfScope ps("embed_sort", st);
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
      OPS_CHECK(launch_dep(k_embed_scatter, dim3(p.blocks), SORT_THREADS, st, s));
    }
  }
  ProfScope ps("embed_grad", st);
  ps.set_kernels(p.levels);
  const bool v4 = a.D % 4 == 0 && a.ld_table % 4 == 0 && a.ld_rows % 4 == 0 &&
                  aligned_to(dtable, 16) && aligned_to(drows, 4 * op_size(dims->row_dtype));
  for (int l = 0; l < p.levels; ++l) {
    SumArgs s{};
    s.n = (int)p.n[l]; s.V = a.V; s.D = a.D;
    s.key = at(l ? p.w_pkey[l - 1] : p.w_key[out]);
    s.idx = at(l ? p.w_pidx[l - 1] : p.w_idx[out]);
    s.ld_src = l ? p.ldp : a.ld_rows;
    s.scale = a.scale;
    s.dtable = dtable; s.ld_table = a.ld_table;
    s.chunks = (int)p.chunks[l];
    s.ldp = p.ldp;
    if (l + 1 < p.levels) {
      s.pkey = at(p.w_pkey[l]);
      s.pidx = at(p.w_pidx[l]);
      s.part = (float*)(w + p.w_part[l]);
    }
    if (l) {
      OPS_CHECK((launch_sum<SUM_WARPS1, float>(s, w + p.w_part[l - 1], (unsigned)s.chunks, v4, st)));
      continue;
    }
    const unsigned blocks = (unsigned)(s.chunks + cdiv(a.V, 8 * SUM_WARPS0));
    if (dims->row_dtype == RNNT_F32)
      OPS_CHECK((launch_sum<SUM_WARPS0, float>(s, drows, blocks, v4, st)));
    else
      OPS_CHECK((launch_sum<SUM_WARPS0, __nv_bfloat16>(s, drows, blocks, v4, st)));
  }
  return RNNT_OK;
}

}  // extern "C"
