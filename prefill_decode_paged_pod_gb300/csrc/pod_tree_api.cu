// pod_tree_api.cu — plan, run and merge of the tree attention (include/pod.h).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <exception>
#include <mutex>
#include <new>
#include <string>
#include <unordered_map>

#include "../../include/pod.h"
#include "pod_device.cuh"
#include "pod_tree.h"
#include "pod_tree_planner.hpp"

void pod_set_last_error(const std::string& msg);

using namespace pod;

struct pod_tree_s {
  PodTreePlanHost plan;
  int dtype = 0, format = 0, hnd = 0, has_sinks = 0;
  float scale_log2 = 0.f, v_scale = 1.f;
  void* workspace = nullptr;
};

namespace {

// Split tiles: o = sum 2^(lse_i - M) o_i / sum over a row's pieces, in a fixed
// order; the sink enters once, here. The partial rows come from L2, and the
// kernel is bound by how many of them are asked for at once. (One warp a row,
// finding its group by bisection, took 30 us for 65536 rows of two pieces. The
// CTA that finishes a tile last merging it on the spot cost the attention loop
// its registers: 419 -> 510 us for 96 block-scaled requests.)
//
// Few pieces: 32 rows a block, 8 threads a row, all pieces of a row in flight.
template <typename T, int D>
POD_DEV void merge_few(const PodTreeParams& P, const int32_t* g, int chunk) {
  constexpr int NV = D / 32;                         // 16-byte runs a thread
  const int nseg = g[TG_NSEG], nrows = g[TG_NROWS], r = chunk * 32 + (threadIdx.x >> 3), l8 = threadIdx.x & 7;
  if (r >= nrows) return;
  const size_t pr0 = (size_t)g[TG_PROW0] + r;
  float w[POD_TREE_FEW];
  float4 v[POD_TREE_FEW][NV];
#pragma unroll
  for (int j = 0; j < POD_TREE_FEW; ++j) {
    w[j] = -INFINITY;
    if (j < nseg) {
      const size_t pr = pr0 + (size_t)j * nrows;
      w[j] = P.part_lse[pr];
#pragma unroll
      for (int k = 0; k < NV; ++k) v[j][k] = reinterpret_cast<const float4*>(P.part_o + pr * D)[l8 + 8 * k];
    }
  }
  const float M = fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])), Ms = M == -INFINITY ? 0.f : M;
  static_assert(POD_TREE_FEW == 4, "the maximum above is over four pieces");
  float wsum = 0.f;
#pragma unroll
  for (int j = 0; j < POD_TREE_FEW; ++j) {
    w[j] = j < nseg ? ex2(w[j] - Ms) : 0.f;
    wsum += w[j];
  }
  const int packed = g[TG_ROW0] + r, head = g[TG_G] * P.G + packed % P.G;
  const size_t out_row = (size_t)(g[TG_QROW0] + packed / P.G) * P.H + head;
  float denom = wsum;
  if (P.sinks) denom += ex2(P.sinks[head] * 1.4426950408889634f - Ms);
  const float inv = wsum == 0.f ? 0.f : 1.f / denom;   // (no keys: 0, whatever the sink)
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < POD_TREE_FEW; ++j)
      if (j < nseg) {
        a.x = fmaf(w[j], v[j][k].x, a.x);
        a.y = fmaf(w[j], v[j][k].y, a.y);
        a.z = fmaf(w[j], v[j][k].z, a.z);
        a.w = fmaf(w[j], v[j][k].w, a.w);
      }
    reinterpret_cast<uint2*>(static_cast<T*>(P.out) + out_row * D)[l8 + 8 * k] =
        make_uint2(Pack<T>::two(a.x * inv, a.y * inv), Pack<T>::two(a.z * inv, a.w * inv));
  }
  if (l8 == 0 && P.lse) P.lse[out_row] = wsum == 0.f ? -INFINITY : M + log2f(wsum);
}

// Many pieces (a long request): two rows a block, four warps a row, each over
// every fourth piece, joined through shared memory.
template <typename T, int D>
POD_DEV void merge_many(const PodTreeParams& P, const int32_t* g, int chunk) {
  constexpr int PER = D / 32, SLICES = 4;
  __shared__ float part[2][SLICES][D];
  __shared__ float sum[2][SLICES];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp >> 2, slice = warp & 3;
  const int nrows = g[TG_NROWS], nseg = g[TG_NSEG], r = chunk * 2 + sub;
  if (chunk * 2 >= nrows) return;
  const bool live = r < nrows;
  const size_t pr0 = (size_t)g[TG_PROW0] + (live ? r : nrows - 1);
  float M = -INFINITY;
  for (int j = lane; j < nseg; j += 32) M = fmaxf(M, P.part_lse[pr0 + (size_t)j * nrows]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float Ms = M == -INFINITY ? 0.f : M;
  float acc[PER] = {};
  float wsum = 0.f;
#pragma unroll 8
  for (int j = slice; j < nseg; j += SLICES) {
    const size_t pr = pr0 + (size_t)j * nrows;
    const float w = ex2(P.part_lse[pr] - Ms);
    wsum += w;
    const float* src = P.part_o + pr * D + lane * PER;
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      const float2 v = *reinterpret_cast<const float2*>(src + i);
      acc[i] = fmaf(w, v.x, acc[i]);
      acc[i + 1] = fmaf(w, v.y, acc[i + 1]);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) part[sub][slice][lane * PER + i] = acc[i];
  if (lane == 0) sum[sub][slice] = wsum;
  __syncthreads();
  if (slice != 0 || !live) return;
  wsum = (sum[sub][0] + sum[sub][1]) + (sum[sub][2] + sum[sub][3]);
  const int packed = g[TG_ROW0] + r, head = g[TG_G] * P.G + packed % P.G;
  const size_t out_row = (size_t)(g[TG_QROW0] + packed / P.G) * P.H + head;
  float denom = wsum;
  if (P.sinks) denom += ex2(P.sinks[head] * 1.4426950408889634f - Ms);
  const float inv = wsum == 0.f ? 0.f : 1.f / denom;   // (no keys: 0, whatever the sink)
  T* out = static_cast<T*>(P.out) + out_row * D + lane * PER;
#pragma unroll
  for (int i = 0; i < PER; i += 2) {
    const int c = lane * PER + i;
    float v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      v[k] = ((part[sub][0][c + k] + part[sub][1][c + k]) + (part[sub][2][c + k] + part[sub][3][c + k])) * inv;
    *reinterpret_cast<uint32_t*>(out + i) = Pack<T>::two(v[0], v[1]);
  }
  if (lane == 0 && P.lse) P.lse[out_row] = wsum == 0.f ? -INFINITY : M + log2f(wsum);
}

constexpr int kManyChunks = POD_TREE_TILE / 2, kFewChunks = POD_TREE_TILE / 32;

template <typename T, int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ PodTreeParams P) {
  // the next call's kernel may set itself up beside this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int many = P.n_big * kManyChunks, b = (int)blockIdx.x;
  if (b < many)
    merge_many<T, D>(P, P.groups + (size_t)(b / kManyChunks) * TG_REC, b % kManyChunks);
  else
    merge_few<T, D>(P, P.groups + (size_t)(P.n_big + (b - many) / kFewChunks) * TG_REC, (b - many) % kFewChunks);
}

template <typename T, int D>
cudaError_t merge_d(const PodTreeParams& P, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const long long blocks = (long long)P.n_big * kManyChunks + (long long)(P.n_groups - P.n_big) * kFewChunks;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<T, D>, P);
}

pod_status fail(pod_status code, const std::string& msg) {
  pod_set_last_error(msg);
  return code;
}
pod_status cuda_fail(cudaError_t e, const char* what) {
  return fail(POD_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

// Which tree plan a workspace holds: the one bound to it last. A run of an earlier one
// would take the other's tables for its own, so it is refused. (Never destroyed:
// handles may outlive static objects.)
struct Owners {
  std::mutex mu;
  std::unordered_map<const void*, pod_tree_handle> of;
};
Owners& owners() {
  static Owners* o = new Owners;
  return *o;
}
void give_up(pod_tree_handle h) {
  std::lock_guard<std::mutex> lock(owners().mu);
  auto it = owners().of.find(h->workspace);
  if (it != owners().of.end() && it->second == h) owners().of.erase(it);
  h->workspace = nullptr;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// The cache as [row part][slot][d / part][Hk][2 * page + kv], a row part 128
// bytes (or the whole row where that is shorter): a box holds `kbx` keys of one
// head, `parts` row parts of them ([part][key][bytes] in shared memory),
// swizzled by the hardware.
CUresult encode(CUtensorMap* m, const void* kv, const PodTreePlanHost& P, int hnd, int kbx, bool whole, int dtype,
                bool f8) {
  const cuuint64_t row = (cuuint64_t)P.d * (f8 ? 1 : 2), ps = P.ps, Hk = P.Hk;
  const cuuint64_t partb = row < 128 ? row : 128, el = partb / (f8 ? 1 : 2), np = row / partb;
  cuuint64_t dims[5] = {el, ps, np, Hk, 2 * (cuuint64_t)P.num_pages};
  cuuint64_t strides[4] = {hnd ? row : row * Hk, partb, hnd ? row * ps : row, row * Hk * ps};
  cuuint32_t box[5] = {(cuuint32_t)el, (cuuint32_t)kbx, whole ? (cuuint32_t)np : 1u, 1, 1}, es[5] = {1, 1, 1, 1, 1};
  return encode_fn()(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                           : dtype ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     5, const_cast<void*>(kv), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     partb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

}  // namespace

void pod_tree_workspace_lost(void* workspace) {
  std::lock_guard<std::mutex> lock(owners().mu);
  owners().of.erase(workspace);
}

cudaError_t pod_tree_merge(const PodTreeParams& P, int dtype, int d, cudaStream_t st) {
  if (dtype == 1)
    return d == 64 ? merge_d<__nv_bfloat16, 64>(P, st)
           : d == 128 ? merge_d<__nv_bfloat16, 128>(P, st)
                      : merge_d<__nv_bfloat16, 256>(P, st);
  return d == 64 ? merge_d<__half, 64>(P, st) : d == 128 ? merge_d<__half, 128>(P, st) : merge_d<__half, 256>(P, st);
}

extern "C" {

pod_status pod_tree_bind_workspace(pod_tree_handle h, void* workspace, size_t workspace_bytes, void* stream) {
  pod_set_last_error("");
  if (!h) return fail(POD_ERR_INVALID_ARG, "handle is NULL");
  const PodTreePlanHost& P = h->plan;
  if (!workspace || workspace_bytes < P.total)
    return fail(POD_ERR_WORKSPACE, "workspace of " + std::to_string(workspace ? workspace_bytes : 0) +
                                       " bytes is smaller than the plan's " + std::to_string(P.total));
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(POD_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  give_up(h);
  pod_tree_workspace_lost(workspace);
  cudaError_t e = cudaMemcpyAsync(workspace, P.image.data(), P.image.size(), cudaMemcpyHostToDevice, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyAsync(tree plan)");
  // the copy reads pageable host memory that the handle owns
  e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize(tree plan)");
  try {
    std::lock_guard<std::mutex> lock(owners().mu);
    owners().of[workspace] = h;
  } catch (const std::exception&) {
    return fail(POD_ERR_INVALID_ARG, "out of host memory");
  }
  h->workspace = workspace;
  return POD_OK;
}

pod_status pod_tree_plan(const int32_t* q_indptr, const int32_t* kv_indptr, const int32_t* kv_indices,
                         const int32_t* last_page_len, int32_t batch, int32_t num_pages, int32_t num_qo_heads,
                         int32_t num_kv_heads, int32_t head_dim, int32_t page_size, float sm_scale, pod_dtype dtype,
                         int32_t kv_format, float k_scale, float v_scale, int32_t kv_layout, int32_t has_sinks,
                         int32_t num_sms, void* workspace, size_t workspace_bytes, void* stream,
                         pod_tree_handle* out_handle, size_t* required_workspace_bytes) {
  pod_set_last_error("");
  if (!out_handle) return fail(POD_ERR_INVALID_ARG, "out_handle is NULL");
  *out_handle = nullptr;
  if (required_workspace_bytes) *required_workspace_bytes = 0;
  if (dtype != POD_F16 && dtype != POD_BF16) return fail(POD_ERR_UNSUPPORTED, "dtype must be fp16 or bf16");
  if (kv_format != POD_KV_16BIT && kv_format != POD_KV_E4M3 && kv_format != POD_KV_E4M3_BLOCK)
    return fail(POD_ERR_INVALID_ARG, "unknown cache format");
  if (kv_layout != 0 && kv_layout != 1) return fail(POD_ERR_INVALID_ARG, "kv_layout must be 0 (NHD) or 1 (HND)");
  if (kv_format == POD_KV_E4M3 && !(k_scale > 0.f && v_scale > 0.f && isfinite(k_scale) && isfinite(v_scale)))
    return fail(POD_ERR_INVALID_ARG, "k_scale and v_scale must be finite and positive");
  if (!isfinite(sm_scale)) return fail(POD_ERR_INVALID_ARG, "sm_scale must be finite");
  if (num_sms <= 0) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(SM count)");
  }
  pod_tree_s* h = new (std::nothrow) pod_tree_s();
  if (!h) return fail(POD_ERR_INVALID_ARG, "out of host memory");
  PodTreeArgs a;
  a.q_indptr = q_indptr; a.kv_indptr = kv_indptr; a.kv_indices = kv_indices; a.last_page_len = last_page_len;
  a.batch = batch; a.num_pages = num_pages; a.H = num_qo_heads; a.Hk = num_kv_heads; a.d = head_dim;
  a.block = kv_format == POD_KV_E4M3_BLOCK ? POD_TREE_BLOCKB : POD_TREE_BLOCK;
  a.ps = page_size; a.slots = num_sms * (head_dim == 256 ? 1 : 2);
  std::string err;
  int rc;
  try {
    rc = pod_tree_build_plan(a, h->plan, &err);
  } catch (const std::exception&) {   // (a vector that cannot grow)
    rc = POD_ERR_INVALID_ARG;
    err = "out of host memory";
  }
  if (rc != POD_OK) {
    delete h;
    return fail((pod_status)rc, err);
  }
  const float scale = sm_scale > 0.f ? sm_scale : 1.f / sqrtf((float)head_dim);
  h->dtype = (int)dtype;
  h->format = kv_format;
  h->hnd = kv_layout;
  h->has_sinks = has_sinks != 0;
  h->scale_log2 = scale * 1.4426950408889634f * (kv_format == POD_KV_E4M3 ? k_scale : 1.f);
  h->v_scale = kv_format == POD_KV_E4M3 ? v_scale : 1.f;
  if (required_workspace_bytes) *required_workspace_bytes = h->plan.total;
  if (workspace) {
    const pod_status st = pod_tree_bind_workspace(h, workspace, workspace_bytes, stream);
    if (st != POD_OK) {
      delete h;
      return st;
    }
  }
  *out_handle = h;
  return POD_OK;
}

size_t pod_tree_workspace_size(pod_tree_handle h) { return h ? h->plan.total : 0; }

pod_status pod_tree_run(pod_tree_handle h, const void* q, const void* kv, const uint8_t* kv_scales,
                        const void* tree_mask, int64_t mask_bytes, const float* sinks, void* workspace, void* out,
                        float* lse, void* stream) {
  pod_set_last_error("");
  if (!h) return fail(POD_ERR_INVALID_ARG, "handle is NULL");
  const PodTreePlanHost& P = h->plan;
  if (!h->workspace) return fail(POD_ERR_WORKSPACE, "the plan has no bound workspace");
  if (workspace != h->workspace) return fail(POD_ERR_WORKSPACE, "workspace differs from the one the plan was bound to");
  {
    std::lock_guard<std::mutex> lock(owners().mu);
    auto it = owners().of.find(workspace);
    if (it == owners().of.end() || it->second != h)
      return fail(POD_ERR_WORKSPACE, "another plan has been bound to the workspace since: bind this one again");
  }
  if (h->has_sinks && !sinks) return fail(POD_ERR_INVALID_ARG, "plan has sinks but sinks is NULL");
  if (!h->has_sinks && sinks) return fail(POD_ERR_INVALID_ARG, "sinks given but the plan was made without sinks");
  if (h->format == POD_KV_E4M3_BLOCK ? !kv_scales : kv_scales != nullptr)
    return fail(POD_ERR_INVALID_ARG, h->format == POD_KV_E4M3_BLOCK ? "a block-scaled cache needs its scales"
                                                                    : "scales given, but the cache format has none");
  if (P.rows == 0) return POD_OK;
  if (!q || !kv || !out) return fail(POD_ERR_INVALID_ARG, "q, kv or out is NULL");
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(kv) | reinterpret_cast<uintptr_t>(out)) & 15u)
    return fail(POD_ERR_INVALID_ARG, "q, kv and out must be 16-byte aligned");
  if (tree_mask && mask_bytes < (P.mask_bits + 7) / 8)
    return fail(POD_ERR_INVALID_ARG, "the tree mask holds " + std::to_string(mask_bytes) + " bytes, the plan needs " +
                                         std::to_string((P.mask_bits + 7) / 8));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PodTreeParams K;
  memset(&K, 0, sizeof(K));
  K.q = q; K.kv = kv; K.scales = kv_scales;
  K.mask = static_cast<const uint8_t*>(tree_mask);
  K.mask_bytes = tree_mask ? mask_bytes : 0;
  K.sinks = sinks; K.out = out; K.lse = lse;
  auto I = [&](size_t off) { return reinterpret_cast<const int32_t*>(ws + off); };
  K.segs = I(P.off_segs); K.cta_ptr = I(P.off_cta); K.pages = I(P.off_pages); K.groups = I(P.off_groups);
  K.part_o = reinterpret_cast<float*>(ws + P.off_part_o);
  K.part_lse = reinterpret_cast<float*>(ws + P.off_part_lse);
  K.status = reinterpret_cast<int32_t*>(ws);
  K.H = P.H; K.Hk = P.Hk; K.G = P.G; K.ps = P.ps; K.hnd = h->hnd; K.num_pages = P.num_pages;
  K.page_rows = 2ll * P.ps * P.Hk;
  K.ps_shift = -1;
  for (int s = 0; s < 31; ++s)
    if ((1 << s) == P.ps) K.ps_shift = s;
  const int block = h->format == POD_KV_E4M3_BLOCK ? POD_TREE_BLOCKB : POD_TREE_BLOCK;
  K.kbx = K.ps_shift >= 3 ? (P.ps < block ? P.ps : block) : 0;
  K.n_cta = P.n_cta; K.n_groups = (int)(P.groups.size() / TG_REC); K.n_big = P.n_big;
  K.scale_log2 = h->scale_log2; K.v_scale = h->v_scale;
  if (K.kbx) {
    if (!encode_fn()) return fail(POD_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const bool f8 = h->format != POD_KV_16BIT;
    CUresult r = encode(&K.tm_k, kv, P, h->hnd, K.kbx, false, h->dtype, f8);
    if (r == CUDA_SUCCESS) r = encode(&K.tm_v, kv, P, h->hnd, K.kbx, !f8, h->dtype, f8);
    if (r != CUDA_SUCCESS) return fail(POD_ERR_CUDA, "cuTensorMapEncodeTiled(tree) failed: " + std::to_string((int)r));
  }
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = h->format == POD_KV_16BIT  ? pod_tree_k16(K, h->dtype, P.d, st)
                  : h->format == POD_KV_E4M3 ? pod_tree_k8(K, h->dtype, P.d, st)
                                             : pod_tree_k8b(K, h->dtype, P.d, st);
  if (e != cudaSuccess) return cuda_fail(e, "tree attention launch");
  if (K.n_groups > 0) {
    e = pod_tree_merge(K, h->dtype, P.d, st);
    if (e != cudaSuccess) return cuda_fail(e, "tree merge launch");
  }
  return POD_OK;
}

pod_status pod_tree_read_device_status(pod_tree_handle h, void* workspace, void* stream, int32_t* device_status) {
  pod_set_last_error("");
  if (!h || !workspace || !device_status) return fail(POD_ERR_INVALID_ARG, "NULL argument");
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, workspace, 4, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e == cudaSuccess && v != 0) e = cudaMemsetAsync(workspace, 0, 4, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "read of the device status");
  *device_status = v;
  return v ? fail(POD_ERR_DEVICE_STATUS, "a kernel recorded device status " + std::to_string(v)) : POD_OK;
}

pod_status pod_tree_plan_table(pod_tree_handle h, int32_t which, int32_t* out, int64_t capacity, int64_t* count) {
  pod_set_last_error("");
  if (!h || !count) return fail(POD_ERR_INVALID_ARG, "NULL argument");
  const PodTreePlanHost& P = h->plan;
  const std::vector<int32_t>* t = which == 0 ? &P.segs : which == 1 ? &P.cta_ptr : which == 2 ? &P.groups
                                  : which == 3 ? &P.pages : nullptr;
  if (!t) return fail(POD_ERR_INVALID_ARG, "unknown table");
  *count = (int64_t)t->size();
  if (out && capacity > 0)
    memcpy(out, t->data(), 4 * (size_t)(capacity < *count ? capacity : *count));
  return POD_OK;
}

pod_status pod_tree_destroy(pod_tree_handle h) {
  if (h) give_up(h);
  delete h;
  return POD_OK;
}

}  // extern "C"
