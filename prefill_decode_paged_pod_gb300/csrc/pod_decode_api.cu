// pod_decode_api.cu — the paged decode's entry points: checks of arguments, the
// workspace, the launches.
#include <cuda_runtime.h>
#include <math.h>

#include <string>

#include "pod_decode.h"

void pod_set_last_error(const std::string& msg);

using namespace pod;

namespace pod {
pod_status check_decode_sizes(const pod_decode_args& a);
pod_status check_decode_cache(const pod_decode_args& a);
pod_status check_decode_rows(const pod_decode_args& a);
}  // namespace pod

namespace {

pod_status fail(pod_status code, const std::string& msg) {
  pod_set_last_error(msg);
  return code;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// The first units of the requests, and for each CTA of the kernel (three an SM, or two that hold
// 16 heads a tile or heads of 256) two pieces of up to four KV heads.
constexpr int kMostCtas = 152 * 3;
size_t piece_rows(int heads, int kv_heads, int d) {
  const bool wide = d < 256 && heads / kv_heads > 8;
  return (size_t)(wide || d == 256 ? 152 * 2 : kMostCtas) * 2 * 4 * (wide ? 16 : 8);
}
size_t first_bytes(int batch) { return round256(8 + (size_t)batch * 8); }

}  // namespace

extern "C" {

size_t pod_paged_decode_workspace_size(int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim) {
  if (batch < 0 || num_kv_heads < 1 || num_qo_heads < 1 || num_qo_heads % num_kv_heads ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  const size_t rows = piece_rows(num_qo_heads, num_kv_heads, head_dim);
  return first_bytes(batch) + round256(rows * sizeof(float2)) + rows * head_dim * 4;
}

pod_status pod_paged_decode(const pod_decode_args* a, void* stream) {
  pod_set_last_error("");
  if (!a) return fail(POD_ERR_INVALID_ARG, "args is NULL");
  pod_status st = check_decode_sizes(*a);
  if (st == POD_OK) st = check_decode_cache(*a);
  if (st == POD_OK) st = check_decode_rows(*a);
  if (st != POD_OK) return st;
  if (a->kv_format == POD_KV_E4M3 && !(a->v_scale > 0.f && isfinite(a->v_scale)))
    return fail(POD_ERR_INVALID_ARG, "k_scale and v_scale must be finite and positive");
  if (!isfinite(a->sm_scale)) return fail(POD_ERR_INVALID_ARG, "sm_scale must be finite");
  if (a->window_left < -1) return fail(POD_ERR_INVALID_ARG, "window_left must be -1 or more");
  if (a->pages && a->num_selected < 1) return fail(POD_ERR_INVALID_ARG, "num_selected must be positive");
  if (a->pages && a->window_left >= 0)
    return fail(POD_ERR_INVALID_ARG, "a window and selected pages do not go together");
  if (!a->batch) return POD_OK;
  if (!a->out || reinterpret_cast<uintptr_t>(a->out) % 16 || a->out_stride % 8 ||
      a->out_stride < (int64_t)a->num_qo_heads * a->head_dim)
    return fail(POD_ERR_INVALID_ARG,
                "out must be 16-byte aligned, its row stride a multiple of 8 elements that holds the row's heads");
  if (!a->workspace || reinterpret_cast<uintptr_t>(a->workspace) % 256 ||
      a->workspace_bytes < pod_paged_decode_workspace_size(a->batch, a->num_qo_heads, a->num_kv_heads, a->head_dim))
    return fail(POD_ERR_WORKSPACE, "the workspace is missing, too small or not 256-byte aligned");
  if ((int64_t)a->batch * a->num_qo_heads > 0x7fffffff) return fail(POD_ERR_INVALID_ARG, "too many rows");
  DecodeParams P = {};
  P.q = a->q;
  P.cache = static_cast<const uint8_t*>(a->kv_cache);
  P.scales = a->kv_scales;
  P.table = a->block_table;
  P.lens = a->kv_lens;
  P.pages = a->pages;
  P.sinks = a->sinks;
  P.out = a->out;
  P.lse = a->lse;
  P.status = a->status;
  char* w = static_cast<char*>(a->workspace);
  P.total = reinterpret_cast<long long*>(w);
  P.first = P.total + 1;
  w += first_bytes(a->batch);
  P.piece_at = reinterpret_cast<float2*>(w);
  w += round256(piece_rows(a->num_qo_heads, a->num_kv_heads, a->head_dim) * sizeof(float2));
  P.piece_o = reinterpret_cast<float*>(w);
  P.q_stride = a->q_stride;
  P.out_stride = a->out_stride;
  P.table_stride = a->table_stride;
  P.num_pages = (unsigned)a->num_pages;
  P.batch = a->batch;
  P.H = a->num_qo_heads;
  P.Hk = a->num_kv_heads;
  P.G = a->num_qo_heads / a->num_kv_heads;
  P.width = a->table_width;
  P.ps = a->page_size;
  P.ps_shift = (P.ps & (P.ps - 1)) == 0 ? __builtin_ctz((unsigned)P.ps) : -1;
  P.hnd = a->kv_layout;
  P.num_selected = a->num_selected;
  P.window = a->window_left;
  const float sm = a->sm_scale > 0.f ? a->sm_scale : 1.f / sqrtf((float)a->head_dim);
  const bool scaled = a->kv_format == POD_KV_E4M3;
  P.scale_log2 = (float)((double)sm * 1.4426950408889634 * (scaled ? (double)a->k_scale : 1.0));
  P.v_scale = scaled ? a->v_scale : 1.f;
  cudaStream_t s = (cudaStream_t)stream;
  const bool bf16 = a->dtype == POD_BF16;
  const cudaError_t e = a->kv_format == POD_KV_16BIT ? decode_launch_16(a->head_dim, bf16, P, s)
                        : scaled                     ? decode_launch_scaled(a->head_dim, bf16, P, s)
                                                     : decode_launch_block(a->head_dim, bf16, P, s);
  if (e != cudaSuccess) return fail(POD_ERR_CUDA, std::string("paged decode launch: ") + cudaGetErrorString(e));
  return POD_OK;
}

}  // extern "C"
