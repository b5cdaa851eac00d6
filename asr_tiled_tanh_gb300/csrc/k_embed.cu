// k_embed.cu -- the prediction network's label embedding (include/rnnt_ops.h).
#include "ops.h"

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

template <typename TE, typename TR>
__global__ void __launch_bounds__(256)
k_embed_rows(EmbedArgs a, const TE* __restrict__ table, TR* __restrict__ rows) {
  const int n = blockIdx.x;
  const int v = label_of(a, n);
  for (int d = threadIdx.x; d < a.D; d += blockDim.x)
    rows[n * a.ld_rows + d] =
        from_f<TR>(v < 0 ? 0.f : a.scale * to_f<TE>(table[v * a.ld_table + d]));
}

// One block per table row: the labels are scanned in order, the rows that
// name it are added in that order.
template <typename TR>
__global__ void __launch_bounds__(256)
k_embed_grad_scan(EmbedArgs a, const TR* __restrict__ drows, float* __restrict__ dtable) {
  __shared__ int lab[256];
  const int v = blockIdx.x, N = a.B * a.U1;
  for (int d0 = 0; d0 < a.D; d0 += blockDim.x) {
    const int d = d0 + threadIdx.x;
    float s = 0.f;
    for (int n0 = 0; n0 < N; n0 += 256) {
      __syncthreads();
      if (n0 + threadIdx.x < N) lab[threadIdx.x] = label_of(a, n0 + threadIdx.x);
      __syncthreads();
      for (int i = 0; i < min(256, N - n0); ++i)
        if (lab[i] == v && d < a.D) s += to_f<TR>(drows[(n0 + i) * a.ld_rows + d]);
    }
    if (d < a.D) dtable[v * a.ld_table + d] = a.scale * s;
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
  return embed_args(dims, &a) ? ALIGN : 0;
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
  const int n = a.B * a.U1;
  using bf = __nv_bfloat16;
  ProfScope ps("embed_rows", st);
  if (dims->table_dtype == RNNT_F32) {
    if (dims->row_dtype == RNNT_F32)
      k_embed_rows<<<n, 256, 0, st>>>(a, (const float*)table, (float*)rows);
    else
      k_embed_rows<<<n, 256, 0, st>>>(a, (const float*)table, (bf*)rows);
  } else {
    if (dims->row_dtype == RNNT_F32)
      k_embed_rows<<<n, 256, 0, st>>>(a, (const bf*)table, (float*)rows);
    else
      k_embed_rows<<<n, 256, 0, st>>>(a, (const bf*)table, (bf*)rows);
  }
  OPS_CHECK(cudaGetLastError());
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
  ProfScope ps("embed_grad", st);
  if (dims->row_dtype == RNNT_F32)
    k_embed_grad_scan<<<a.V, 256, 0, st>>>(a, (const float*)drows, dtable);
  else
    k_embed_grad_scan<<<a.V, 256, 0, st>>>(a, (const __nv_bfloat16*)drows, dtable);
  OPS_CHECK(cudaGetLastError());
  return RNNT_OK;
}

}  // extern "C"
