// pod_step.cu — the start of a decode step whose tables live on the device: pages
// taken from and returned to a free stack, positions and slots of the new tokens,
// the page table end to end.
//
// Mathematics. A request with L keys that gets n more needs
// ceil((L + n) / ps) - ceil(L / ps) pages; prefix sums over the requests give
// every one its place on the stack, in the rows and in the page table. The sums
// are 64 bits wide, so no lengths can wrap them.
//
// Work split. The prefix sums depend on all requests, so one block makes them, a thread
// a request (in rounds past its threads), and moves the pages, a thread a page. Where
// the step may have many rows, or the page table is asked for, a second kernel
// of many blocks writes them (a thread an entry, which finds its request by bisection
// of the offsets); otherwise the first block does it too and the launch is spared.
// Bound by latency: a chain of some ten trips to L2 and as many block barriers. Measured on
// a GB300, in graphs: 64 requests of one token 3.6 us; 768 requests, prompts and tokens
// given back among them (some 14000 pages moved, 80000 rows, 400000 page-table entries) 23 us,
// of which the one block's bisections and moves take 15.
#include <cuda_runtime.h>
#include <limits.h>

#include <string>

#include "../../include/pod.h"
#include "pod_beside.h"
#include "pod_decode.h"
#include "pod_device.cuh"

void pod_set_last_error(const std::string& msg);

using namespace pod;

namespace {

constexpr int kStepThreads = 1024;
constexpr int kRowThreads = 256;
constexpr int kInFlight = 4;       // pages that a thread moves at a time

struct StepParams {
  int32_t* table;
  const int32_t* lens;
  const int32_t* news;
  int32_t* lens_out;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* q_indptr;
  int32_t* requests;
  int32_t* positions;
  int64_t* slots;
  int32_t* kv_indptr;
  int32_t* kv_indices;
  int32_t* last_page_len;
  int32_t* status;
  long long table_stride;
  int batch, width, ps, capacity, max_rows, max_pages, rows_here;
};

// Sums of x[0..N) over the threads before this one (in place), and over all of them.
template <int N>
POD_DEV void block_scan(long long* x, long long* all, long long (*sh)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i] = x[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, s[i], o);
      if (lane >= o) s[i] += y;
    }
  }
  __syncthreads();                                 // (sh may still be read)
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < N; ++i) sh[warp][i] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const long long w = lane < warps ? sh[lane][i] : 0;
    long long t = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    all[i] = __shfl_sync(0xffffffffu, t, 31);
    x[i] = s[i] - x[i] + __shfl_sync(0xffffffffu, t - w, warp);
  }
}

struct Step {
  int old, now;                                    // keys before and after
  int had, has;                                    // their pages
  bool wants;                                      // grows
  int status;                                      // bits for a length out of range, or past its row
};
POD_DEV int pages_for(const StepParams& P, int keys) { return (int)(((unsigned)keys + P.ps - 1) / (unsigned)P.ps); }
POD_DEV Step step_of(const StepParams& P, int len, int n) {
  Step s;
  const int most = P.width * P.ps;                 // (at most 2^30)
  s.old = min(max(len, 0), most);
  s.status = len != s.old ? kStatusSlot : 0;
  const long long now = max(0ll, (long long)s.old + n);
  s.wants = n > 0 && now <= most;
  if (now > most) s.status |= kStatusNoRoom;
  s.now = now > most ? s.old : (int)now;
  s.had = pages_for(P, s.old);
  s.has = pages_for(P, s.now);
  return s;
}

// last i < n with at[i] <= x (at ascending from at[0] <= x)
POD_DEV int find_row(const int32_t* at, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

POD_DEV void write_row(const StepParams& P, int i, int rows, const int32_t* indptr, const int32_t* lens_out) {
  int req = -1, pos = 0;
  long long slot = -1;
  if (i < rows) {
    req = find_row(indptr, P.batch, i);
    pos = lens_out[req] - (indptr[req + 1] - i);
    const int at = pos / P.ps, page = P.table[req * P.table_stride + at];
    if (page >= 0) slot = (long long)page * P.ps + (pos - at * P.ps);
  }
  P.requests[i] = req;
  P.positions[i] = pos;
  P.slots[i] = slot;
}

__global__ void __launch_bounds__(kStepThreads) step_kernel(const __grid_constant__ StepParams P) {
  __shared__ long long sh1[32][1], sh3[32][3];
  __shared__ int sh_off[kStepThreads], sh_first[kStepThreads];   // of the round's requests: pages before, first page moved
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, T = blockDim.x;
  const long long count = min(max((long long)*P.free_count, 0ll), (long long)P.capacity);
  int bad = 0;                                     // status bits
  // ---- pages of shrinking requests go onto the stack
  long long given = 0;
  for (int base = 0; base < P.batch; base += T) {
    const int r = base + tid;
    int n = 0, first = 0;
    if (r < P.batch) {
      const Step s = step_of(P, P.lens[r], P.news[r]);
      n = max(0, s.had - s.has);
      first = s.has;
    }
    if (!__syncthreads_or(n)) continue;            // (most steps take nothing back)
    long long x[1] = {n}, all[1];
    block_scan<1>(x, all, sh1);
    // (a round gives back more than 2^31 pages only where the stack is long full)
    sh_off[tid] = (int)min(x[0], 0x7fffffffll);
    sh_first[tid] = first;
    __syncthreads();
    // (unsigned: an index a few rounds past the last page stays past it)
    const unsigned moved = (unsigned)min(all[0], max(0ll, P.capacity - count - given));
    if (moved < all[0]) bad |= kStatusNoRoom;
    const int32_t* from[kInFlight];
    for (unsigned i = tid; i < moved; i += T * kInFlight) {   // a thread a page, some at a time
      int32_t page[kInFlight];
#pragma unroll
      for (int j = 0; j < kInFlight; ++j)
        if (i + j * T < moved) {
          const int k = find_row(sh_off, T, i + j * T);
          from[j] = P.table + (long long)(base + k) * P.table_stride + sh_first[k] + (int)(i + j * T - sh_off[k]);
        }
#pragma unroll
      for (int j = 0; j < kInFlight; ++j)
        if (i + j * T < moved) page[j] = *from[j];
#pragma unroll
      for (int j = 0; j < kInFlight; ++j)
        if (i + j * T < moved) P.free_pages[count + given + i + j * T] = page[j];
    }
    given += all[0];
  }
  const long long top = min(count + given, (long long)P.capacity);
  // ---- growing requests take theirs off its top (pages pushed above are seen behind
  // the barriers of the scans)
  long long pages = 0, rows = 0, kv = 0, pages_taken = 0, rows_taken = 0;
  for (int base = 0; base < P.batch; base += T) {
    const int r = base + tid;
    Step s = {};
    if (r < P.batch) s = step_of(P, P.lens[r], P.news[r]);
    bad |= s.status;
    const int need = s.wants ? s.has - s.had : 0, n = s.wants ? s.now - s.old : 0;
    // pages and rows asked for, and the pages of all, each as sums over the requests before
    long long x[3] = {need, n, s.has}, all[3];
    block_scan<3>(x, all, sh3);
    long long y[3] = {x[0], x[1], x[2]}, sums[3] = {all[0], all[1], all[2]};   // of those that are granted
    const long long p0 = pages + x[0], r0 = rows + x[1];
    if (pages + all[0] > top || rows + all[1] > P.max_rows) {
      // (the granted ones come before every refused one)
      const bool granted = s.wants && p0 + need <= top && r0 + n <= P.max_rows;
      if (s.wants && !granted) {
        bad |= kStatusNoRoom;
        s.now = s.old;
        s.has = s.had;
      }
      y[0] = granted ? need : 0;
      y[1] = granted ? n : 0;
      y[2] = s.has;
      block_scan<3>(y, sums, sh3);
    }
    rows_taken += sums[1];
    if (r < P.batch) {
      P.lens_out[r] = s.now;
      P.q_indptr[r + 1] = (int)min(r0 + n, rows_taken);
      if (P.kv_indptr) {
        P.kv_indptr[r + 1] = (int)min(kv + y[2] + s.has, (long long)INT_MAX);
        P.last_page_len[r] = s.now ? (int)((unsigned)(s.now - 1) % (unsigned)P.ps) + 1 : 0;
      }
    }
    sh_off[tid] = (int)y[0];
    sh_first[tid] = s.had;
    __syncthreads();
    const unsigned taken = (unsigned)sums[0];
    for (unsigned i = tid; i < taken; i += T * kInFlight) {
      int32_t page[kInFlight];
#pragma unroll
      for (int j = 0; j < kInFlight; ++j)
        if (i + j * T < taken) page[j] = P.free_pages[top - 1 - pages_taken - i - j * T];
#pragma unroll
      for (int j = 0; j < kInFlight; ++j)
        if (i + j * T < taken) {
          const int k = find_row(sh_off, T, i + j * T);
          P.table[(long long)(base + k) * P.table_stride + sh_first[k] + (int)(i + j * T - sh_off[k])] = page[j];
        }
    }
    pages += all[0];
    rows += all[1];
    kv += sums[2];
    pages_taken += sums[0];
    __syncthreads();                               // (the arrays are the next round's)
  }
  if (P.kv_indptr && kv > P.max_pages) bad |= kStatusNoRoom;
  if (tid == 0) {
    *P.free_count_out = (int)(top - pages_taken);
    P.q_indptr[0] = 0;
    if (P.kv_indptr) P.kv_indptr[0] = 0;
  }
  if (__syncthreads_or(bad) && P.status) {         // (the rows below read what the block wrote above)
    const int bits = __reduce_or_sync(0xffffffffu, bad);
    if ((tid & 31) == 0 && bits) atomicOr(P.status, bits);
  }
  if (P.rows_here)
    for (int i = tid; i < P.max_rows; i += T) write_row(P, i, (int)rows_taken, P.q_indptr, P.lens_out);
}

// rows first, then entries of the page table
__global__ void __launch_bounds__(kRowThreads) step_rows_kernel(const __grid_constant__ StepParams P) {
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const long long stride = (long long)gridDim.x * kRowThreads, n = (long long)P.max_rows + (P.kv_indptr ? P.max_pages : 0);
  const int rows = P.q_indptr[P.batch], pages = P.kv_indptr ? P.kv_indptr[P.batch] : 0;
  for (long long i = (long long)blockIdx.x * kRowThreads + threadIdx.x; i < n; i += stride) {
    if (i < P.max_rows) {
      write_row(P, (int)i, rows, P.q_indptr, P.lens_out);
    } else {
      const int j = (int)(i - P.max_rows);
      int page = -1;
      if (j < pages) {
        const int r = find_row(P.kv_indptr, P.batch, j);
        page = P.table[r * P.table_stride + j - P.kv_indptr[r]];
      }
      P.kv_indices[j] = page;
    }
  }
}

pod_status fail(pod_status code, const std::string& msg) {
  pod_set_last_error(msg);
  return code;
}

}  // namespace

extern "C" pod_status pod_step_tables(const pod_step_args* a, void* stream) {
  pod_set_last_error("");
  if (!a) return fail(POD_ERR_INVALID_ARG, "args is NULL");
  if (a->batch < 0 || a->max_rows < 0 || a->max_pages < 0 || a->free_capacity < 0)
    return fail(POD_ERR_INVALID_ARG, "batch, max_rows, max_pages and free_capacity must not be negative");
  if (a->page_size < 1 || a->table_width < 1 || (int64_t)a->table_width * a->page_size > (1 << 30))
    return fail(POD_ERR_INVALID_ARG, "table_width and page_size must be positive, their product at most 2^30");
  if (a->batch > 1 && a->table_stride < a->table_width)
    return fail(POD_ERR_INVALID_ARG, "table_stride must hold table_width entries");
  if (!a->free_count || !a->free_count_out || !a->q_indptr ||
      (a->batch && (!a->block_table || !a->kv_lens || !a->new_lens || !a->kv_lens_out)) ||
      (a->free_capacity && !a->free_pages) || (a->max_rows && (!a->requests || !a->positions || !a->slots)))
    return fail(POD_ERR_INVALID_ARG, "an array is NULL");
  if ((a->batch && !a->kv_indptr != !a->last_page_len) || (a->kv_indptr && a->max_pages && !a->kv_indices))
    return fail(POD_ERR_INVALID_ARG, "kv_indptr, kv_indices and last_page_len come together");
  StepParams P = {};
  P.table = a->block_table;
  P.lens = a->kv_lens;
  P.news = a->new_lens;
  P.lens_out = a->kv_lens_out;
  P.free_pages = a->free_pages;
  P.free_count = a->free_count;
  P.free_count_out = a->free_count_out;
  P.q_indptr = a->q_indptr;
  P.requests = a->requests;
  P.positions = a->positions;
  P.slots = a->slots;
  P.kv_indptr = a->kv_indptr;
  P.kv_indices = a->kv_indices;
  P.last_page_len = a->last_page_len;
  P.status = a->status;
  P.table_stride = a->table_stride;
  P.batch = a->batch;
  P.width = a->table_width;
  P.ps = a->page_size;
  P.capacity = a->free_capacity;
  P.max_rows = a->max_rows;
  P.max_pages = a->max_pages;
  cudaStream_t st = (cudaStream_t)stream;
  const int threads = a->batch <= 128 ? 128 : a->batch >= kStepThreads ? kStepThreads : (a->batch + 31) / 32 * 32;
  // No more rows than threads: the first block writes them (64 requests of one token 3.6 us,
  // by a second kernel 5.2; 1024 of them 6.6 and 8.5; 8 requests with 2048 rows 10.2 and 4.8).
  P.rows_here = !a->kv_indptr && a->max_rows <= threads;
  cudaError_t e = launch_beside(step_kernel, 1, (unsigned)threads, 0, 1, st, P);
  const int64_t entries = (int64_t)a->max_rows + (a->kv_indptr ? a->max_pages : 0);
  if (e == cudaSuccess && !P.rows_here && entries) {
    const int64_t blocks = (entries + kRowThreads - 1) / kRowThreads;
    e = launch_beside(step_rows_kernel, (unsigned)(blocks < 152 * 8 ? blocks : 152 * 8), kRowThreads, 0, 1, st,
                      P);
  }
  if (e != cudaSuccess) return fail(POD_ERR_CUDA, std::string("step tables launch: ") + cudaGetErrorString(e));
  return POD_OK;
}
