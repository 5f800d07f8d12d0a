// Embedding lookup with a scale, and its gradient by sorted ids.
//
// A table of K rows shared by n items (a colour codebook shared by the
// Gaussians, a per-view embedding): out[j] = scale * table[id_j], and
//   dtable[k] = scale * sum over {j : id_j = k} of g[j].
// gs_grad_accumulate scatters gradients whose indices are all different;
// here an index may occur any number of times, so the rows are first sorted
// by id (the library's stable radix sort) and each run of equal ids is
// summed in order: no float atomics, the same result on every call.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gs_internal.cuh"

namespace gs {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kNoRow = 0xffffffffu;  // key of an unused partial

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// The id of item j: ids[index[j]] or ids[j]; -1 for "no row", also for an
// index or id out of range (which is flagged).
__device__ __forceinline__ int32_t id_of(const int32_t* __restrict__ ids, int64_t n_ids,
                                         const int32_t* __restrict__ index, int64_t j, int64_t rows,
                                         int32_t* dev_status) {
  int64_t at = j;
  if (index) {
    at = index[j];
    if (at < 0 || at >= n_ids) {
      dev_flag(dev_status, GS_DEV_BOUNDS);
      return -1;
    }
  }
  const int32_t id = ids[at];
  if (id >= rows) {
    dev_flag(dev_status, GS_DEV_BOUNDS);
    return -1;
  }
  return id;
}

// One thread per element of out; the contiguous axis of out runs fastest.
template <class TT, class TO>
__global__ void __launch_bounds__(kThreads)
k_lookup(const TT* __restrict__ table, int64_t ld, int64_t rows, const int32_t* __restrict__ ids,
         int64_t n_ids, const int32_t* __restrict__ index, float scale, TO* __restrict__ out,
         int64_t n, int cols, int64_t rs, int64_t cs, int32_t* dev_status) {
  const int64_t total = n * cols, step = (int64_t)gridDim.x * kThreads;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < total; e += step) {
    const int64_t j = cs == 1 ? e / cols : e % n;
    const int64_t c = cs == 1 ? e % cols : e / n;
    const int32_t id = id_of(ids, n_ids, index, j, rows, dev_status);
    const float v = id >= 0 ? scale * to_f(table[(int64_t)id * ld + c]) : 0.f;
    out[j * rs + c * cs] = from_f<TO>(v);
  }
}

// Sort keys and values of the gradient's items: key = id, value = j.  An
// item without a row takes the last key and a negative value, which adds
// nothing, so that the keys need no bit more than the rows do.
__global__ void __launch_bounds__(kThreads)
k_lookup_keys(const int32_t* __restrict__ ids, int64_t n_ids, const int32_t* __restrict__ index,
              int64_t n, int64_t rows, uint32_t* __restrict__ keys, int32_t* __restrict__ vals,
              int32_t* dev_status) {
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= n) return;
  const int32_t id = id_of(ids, n_ids, index, j, rows, dev_status);
  keys[j] = id >= 0 ? (uint32_t)id : (uint32_t)(rows - 1);
  vals[j] = id >= 0 ? (int32_t)j : -1;
}

// Sums of runs of equal keys over a list of n entries, entry r standing for
// the row order[r] of g (or row r).  The list is cut into chunks of R
// entries; a thread sums one column of one chunk in order.  A run that lies
// inside a chunk goes to dtable.  What a chunk holds of a run that goes on
// across its border is a partial: entry 2 chunk for a run that came in from
// the chunk before, 2 chunk + 1 for one that starts here and goes on.  A
// chunk inside one run writes its sum at 2 chunk and zeros at 2 chunk + 1,
// so that the partials of one run are neighbours; unused partials have the
// key kNoRow.  The partials are summed by the same kernel.
template <class T>
__global__ void __launch_bounds__(kThreads)
k_run_sums(const uint32_t* __restrict__ keys, const int32_t* __restrict__ order, int64_t n, int R,
           const T* __restrict__ g, int64_t rs, int64_t cs, int cols, float scale,
           float* __restrict__ dtable, int64_t ld, bool accumulate, uint32_t* __restrict__ pkey,
           float* __restrict__ psum) {
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t chunk = e / cols;
  const int c = (int)(e % cols);
  const int64_t a = chunk * R;
  if (a >= n) return;
  const int64_t b = min(a + R, n);
  uint32_t k = keys[a];
  bool head = a > 0 && keys[a - 1] == k;  // the run came in from the chunk before
  bool used0 = false, used1 = false;
  float sum = 0.f;
  auto done = [&](bool tail) {
    if (k == kNoRow) return;
    if (head || tail) {
      const int64_t at = 2 * chunk + (head ? 0 : 1);
      psum[at * cols + c] = sum;
      if (c == 0) pkey[at] = k;
      (head ? used0 : used1) = true;
      if (head && tail) {
        psum[(at + 1) * cols + c] = 0.f;
        if (c == 0) pkey[at + 1] = k;
        used1 = true;
      }
    } else {
      float* d = dtable + (int64_t)k * ld + c;
      *d = accumulate ? *d + scale * sum : scale * sum;
    }
  };
  for (int64_t r = a; r < b; ++r) {
    const uint32_t kr = keys[r];
    if (kr != k) {
      done(false);
      k = kr;
      head = false;
      sum = 0.f;
    }
    const int64_t j = order ? order[r] : r;
    if (k != kNoRow && j >= 0) sum += to_f(g[j * rs + (int64_t)c * cs]);
  }
  done(b < n && keys[b] == k);
  if (c == 0 && pkey) {
    if (!used0) pkey[2 * chunk] = kNoRow;
    if (!used1) pkey[2 * chunk + 1] = kNoRow;
  }
}

int key_bits(int64_t rows) { return rows > 1 ? 64 - __builtin_clzll((unsigned long long)(rows - 1)) : 0; }

constexpr int kChunk = 64;  // entries per chunk

struct LookupWs {
  uint32_t* keys;
  int32_t* order;
  void* sort;
  size_t sort_bytes;
  uint32_t* pkey[2];
  float* psum[2];
  size_t bytes;
};

LookupWs carve_lookup(void* ws, size_t cap, int64_t n, int64_t rows, int cols) {
  LookupWs w{};
  Carver cv(ws, cap);
  w.keys = cv.take<uint32_t>(n);
  w.order = cv.take<int32_t>(n);
  w.sort_bytes = gs_sort_workspace_size(n, 4, 0, key_bits(rows));
  w.sort = cv.take<char>(w.sort_bytes);
  int64_t m = 2 * ((n + kChunk - 1) / kChunk);
  for (int k = 0; k < 2; ++k) {
    w.pkey[k] = cv.take<uint32_t>(m);
    w.psum[k] = cv.take<float>((size_t)m * cols);
    m = 2 * ((m + kChunk - 1) / kChunk);
  }
  w.bytes = cv.off;
  return w;
}

size_t type_size(int dtype) { return dtype == GS_F32 ? 4 : dtype == GS_F16 || dtype == GS_BF16 ? 2 : 0; }

// A matrix whose elements do not overlap: one stride is 1, the other spans
// at least the extent of the contiguous axis.
bool good_matrix(const gs_matrix* m) {
  if (!m || m->rows < 0 || m->cols < 1 || !type_size(m->dtype)) return false;
  if (m->rows == 0) return true;
  if (!m->data || !aligned(m->data, type_size(m->dtype))) return false;
  if (m->col_stride == 1) return m->row_stride >= m->cols;
  return m->row_stride == 1 && m->col_stride >= m->rows;
}

gs_status check_ids(const int32_t* ids, int64_t n_ids, const int32_t* index, int64_t n) {
  if (n < 0 || n_ids < 0) return GS_ERR_ARG;
  if (n > (int64_t)INT32_MAX) return GS_ERR_UNSUPPORTED;  // positions are int32
  if (n > 0 && ((!ids && n_ids > 0) || (!index && n_ids < n))) return GS_ERR_ARG;
  if (!aligned(ids, 4) || !aligned(index, 4)) return GS_ERR_ARG;
  return GS_OK;
}

unsigned blocks_for(int64_t threads) { return (unsigned)((threads + kThreads - 1) / kThreads); }

gs_status plan_lookup(const int32_t* ids, int64_t n_ids, const int32_t* index, int64_t n,
                      int64_t rows, const LookupWs& w, int32_t* dev_status, cudaStream_t s) {
  k_lookup_keys<<<blocks_for(n), kThreads, 0, s>>>(ids, n_ids, index, n, rows, w.keys, w.order,
                                                   dev_status);
  GS_LAUNCH_CHECK();
  return gs_sort_keys32(nullptr, w.keys, w.order, n, 0, key_bits(rows), 0, w.sort, w.sort_bytes,
                        dev_status, s);
}

template <class T>
gs_status run_sums(const gs_matrix* g, const gs_matrix* dtable, float scale, bool accumulate,
                   const LookupWs& w, cudaStream_t s) {
  const int cols = g->cols;
  float* dt = static_cast<float*>(dtable->data);
  int64_t m = g->rows, chunks = (m + kChunk - 1) / kChunk;
  k_run_sums<T><<<blocks_for(chunks * cols), kThreads, 0, s>>>(
      w.keys, w.order, m, kChunk, static_cast<const T*>(g->data), g->row_stride, g->col_stride, cols,
      scale, dt, dtable->row_stride, accumulate, w.pkey[0], w.psum[0]);
  GS_LAUNCH_CHECK();
  for (int from = 0; chunks > 1; from ^= 1) {
    m = 2 * chunks;
    chunks = (m + kChunk - 1) / kChunk;
    k_run_sums<float><<<blocks_for(chunks * cols), kThreads, 0, s>>>(
        w.pkey[from], nullptr, m, kChunk, w.psum[from], cols, 1, cols, scale, dt,
        dtable->row_stride, accumulate, w.pkey[from ^ 1], w.psum[from ^ 1]);
    GS_LAUNCH_CHECK();
  }
  return GS_OK;
}

template <class TT, class TO>
gs_status launch_lookup(const gs_matrix* t, const int32_t* ids, int64_t n_ids, const int32_t* index,
                        float scale, const gs_matrix* o, int32_t* dev_status, cudaStream_t s) {
  const int64_t blocks = (o->rows * o->cols + kThreads - 1) / kThreads;
  k_lookup<TT, TO><<<(unsigned)(blocks < 148 * 64 ? blocks : 148 * 64), kThreads, 0, s>>>(
      static_cast<const TT*>(t->data), t->row_stride, t->rows, ids, n_ids, index, scale,
      static_cast<TO*>(o->data), o->rows, o->cols, o->row_stride, o->col_stride, dev_status);
  GS_LAUNCH_CHECK();
  return GS_OK;
}

template <class TT>
gs_status lookup_to(const gs_matrix* t, const int32_t* ids, int64_t n_ids, const int32_t* index,
                    float scale, const gs_matrix* o, int32_t* dev_status, cudaStream_t s) {
  switch (o->dtype) {
    case GS_F32: return launch_lookup<TT, float>(t, ids, n_ids, index, scale, o, dev_status, s);
    case GS_F16: return launch_lookup<TT, __half>(t, ids, n_ids, index, scale, o, dev_status, s);
    default: return launch_lookup<TT, __nv_bfloat16>(t, ids, n_ids, index, scale, o, dev_status, s);
  }
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" gs_status gs_lookup(const gs_matrix* table, const int32_t* ids, int64_t n_ids,
                               const int32_t* index, double scale, const gs_matrix* out,
                               int32_t* dev_status, gs_stream stream) {
  if (!good_matrix(table) || !good_matrix(out) || table->cols != out->cols) return GS_ERR_ARG;
  const gs_status st = check_ids(ids, n_ids, index, out->rows);
  if (st != GS_OK) return st;
  if (out->rows == 0) return GS_OK;
  if (table->rows < 1) return GS_ERR_ARG;
  if (table->col_stride != 1) return GS_ERR_UNSUPPORTED;  // a table's rows are contiguous
  const float sc = (float)scale;
  cudaStream_t s = to_stream(stream);
  switch (table->dtype) {
    case GS_F32: return lookup_to<float>(table, ids, n_ids, index, sc, out, dev_status, s);
    case GS_F16: return lookup_to<__half>(table, ids, n_ids, index, sc, out, dev_status, s);
    default: return lookup_to<__nv_bfloat16>(table, ids, n_ids, index, sc, out, dev_status, s);
  }
}

extern "C" size_t gs_lookup_bwd_workspace_size(int64_t n, int64_t rows, int32_t cols,
                                               int32_t planes) {
  (void)planes;
  if (n < 0 || n > (int64_t)INT32_MAX || rows < 1 || cols < 1) return 0;
  return carve_lookup(nullptr, 0, n, rows, cols).bytes;
}

extern "C" gs_status gs_lookup_plan(const int32_t* ids, int64_t n_ids, const int32_t* index,
                                    int64_t n, int64_t rows, int32_t cols, void* ws, size_t ws_bytes,
                                    int32_t* dev_status, gs_stream stream) {
  const gs_status st = check_ids(ids, n_ids, index, n);
  if (st != GS_OK) return st;
  if (rows < 1 || rows > (int64_t)INT32_MAX || cols < 1) return GS_ERR_ARG;
  if (n == 0) return GS_OK;
  const LookupWs w = carve_lookup(ws, ws_bytes, n, rows, cols);
  if (!ws || w.bytes > ws_bytes) return GS_ERR_CAPACITY;
  if (!aligned(ws, 256)) return GS_ERR_ARG;
  return plan_lookup(ids, n_ids, index, n, rows, w, dev_status, to_stream(stream));
}

extern "C" gs_status gs_lookup_bwd(const gs_matrix* g, const int32_t* ids, int64_t n_ids,
                                   const int32_t* index, double scale, const gs_matrix* dtable,
                                   uint32_t flags, void* ws, size_t ws_bytes, int32_t* dev_status,
                                   gs_stream stream) {
  if (flags & ~(GS_LOOKUP_ACCUMULATE | GS_LOOKUP_PLANNED)) return GS_ERR_ARG;
  if (!good_matrix(g) || !good_matrix(dtable) || g->cols != dtable->cols) return GS_ERR_ARG;
  if (dtable->rows < 1 || dtable->rows > (int64_t)INT32_MAX) return GS_ERR_ARG;
  if (dtable->dtype != GS_F32 || dtable->col_stride != 1) return GS_ERR_UNSUPPORTED;
  const int64_t n = g->rows, rows = dtable->rows;
  const gs_status st = check_ids(ids, n_ids, index, n);
  if (st != GS_OK) return st;
  cudaStream_t s = to_stream(stream);
  const LookupWs w = carve_lookup(ws, ws_bytes, n, rows, g->cols);
  if (n > 0) {
    if (!ws || w.bytes > ws_bytes) return GS_ERR_CAPACITY;
    if (!aligned(ws, 256)) return GS_ERR_ARG;
  }
  const bool accumulate = (flags & GS_LOOKUP_ACCUMULATE) != 0;
  if (!accumulate)
    GS_TRY(cudaMemset2DAsync(dtable->data, dtable->row_stride * 4, 0, (size_t)g->cols * 4, rows, s));
  if (n == 0) return GS_OK;
  if (!(flags & GS_LOOKUP_PLANNED)) {
    const gs_status ps = plan_lookup(ids, n_ids, index, n, rows, w, dev_status, s);
    if (ps != GS_OK) return ps;
  }
  const float sc = (float)scale;
  switch (g->dtype) {
    case GS_F32: return run_sums<float>(g, dtable, sc, accumulate, w, s);
    case GS_F16: return run_sums<__half>(g, dtable, sc, accumulate, w, s);
    default: return run_sums<__nv_bfloat16>(g, dtable, sc, accumulate, w, s);
  }
}
