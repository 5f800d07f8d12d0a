// The global gradient norm over many tensors, clipping, and Adam on the
// clipped gradient.
//
//   N = sqrt(sum over all elements of g^2),   c = min(1, max_norm / (N + eps))
//   clipped g = c g,   Adam on c g.
// The norm is a sum over everything before anything can be scaled, so the
// coefficient stays on the device: Adam (or the clipping copy) reads it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "gs_internal.cuh"

namespace gs {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 8192;      // elements a block takes at a time
constexpr int kMaxTensors = 256;  // tensors per launch, passed by value
constexpr int kNormBlocks = 148 * 4;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

struct Entry {
  const void* src;
  void* dst;
  int64_t cols, src_stride, dst_stride, size;  // size = rows * cols
  int64_t unit0;                               // first unit of this tensor
  int32_t dtype;
};

struct Table {
  Entry t[kMaxTensors];
  int32_t count;
  int64_t units;
};

// Calls f(typed src, typed dst, element offset in src, in dst) for this
// thread's elements of unit u.
template <class T, class F>
__device__ __forceinline__ void unit_elements(const Entry& e, int64_t u, F&& f) {
  const T* src = static_cast<const T*>(e.src);
  T* dst = static_cast<T*>(e.dst);
  const int64_t a = (u - e.unit0) * kUnit, b = min(a + kUnit, e.size);
  for (int64_t i = a + threadIdx.x; i < b; i += kThreads) {
    const int64_t r = i / e.cols, c = i - r * e.cols;
    f(src, dst, r * e.src_stride + c, r * e.dst_stride + c);
  }
}

template <class F>
__device__ __forceinline__ void each_unit(const Table& tab, F&& f) {
  for (int64_t u = blockIdx.x; u < tab.units; u += gridDim.x) {
    int lo = 0, hi = tab.count - 1;  // the last tensor with unit0 <= u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.t[mid].unit0 <= u) lo = mid;
      else hi = mid - 1;
    }
    const Entry& e = tab.t[lo];
    f(e, u);
  }
}

// Sums of squares in fp64: a square of a finite fp32 value neither overflows
// nor vanishes there, and a sum over 2^40 elements keeps 1e-4 of its last
// fp32 place.
__global__ void __launch_bounds__(kThreads)
k_sum_squares(const __grid_constant__ Table tab, double* __restrict__ part) {
  __shared__ double s_warp[kThreads / 32];
  double sum = 0.0;
  each_unit(tab, [&](const Entry& e, int64_t u) {
    auto add = [&](auto* src, auto*, int64_t at, int64_t) {
      const double x = (double)to_f(src[at]);
      sum = fma(x, x, sum);
    };
    if (e.dtype == GS_F32) unit_elements<float>(e, u, add);
    else if (e.dtype == GS_F16) unit_elements<__half>(e, u, add);
    else unit_elements<__nv_bfloat16>(e, u, add);
  });
  sum = warp_sum(sum);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) sum += s_warp[w];
    part[blockIdx.x] = sum;
  }
}

// clip[0] = norm, clip[1] = coefficient (see gs.h for non-finite norms)
__global__ void __launch_bounds__(kThreads)
k_clip_coef(const double* __restrict__ part, int n, double max_norm, double eps,
            float* __restrict__ clip, int32_t* dev_status) {
  __shared__ double s_warp[kThreads / 32];
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) sum += part[i];
  sum = warp_sum(sum);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) sum += s_warp[w];
    const double norm = sqrt(sum);
    const double c = max_norm / (norm + eps);
    clip[0] = (float)norm;
    clip[1] = (float)(c < 1.0 ? c : isnan(norm) ? norm : 1.0);
    if (!isfinite(norm)) dev_flag(dev_status, GS_DEV_NONFINITE);
  }
}

__global__ void __launch_bounds__(kThreads)
k_clip(const __grid_constant__ Table tab, const float* __restrict__ clip) {
  const float c = clip[1];
  each_unit(tab, [&](const Entry& e, int64_t u) {
    if (c == 1.0f && e.src == e.dst) return;  // in place and nothing to clip
    auto scale = [&](auto* src, auto* dst, int64_t at, int64_t to) { put(dst + to, c * to_f(src[at])); };
    if (e.dtype == GS_F32) unit_elements<float>(e, u, scale);
    else if (e.dtype == GS_F16) unit_elements<__half>(e, u, scale);
    else unit_elements<__nv_bfloat16>(e, u, scale);
  });
}

size_t type_size(int dtype) { return dtype == GS_F32 ? 4 : dtype == GS_F16 || dtype == GS_BF16 ? 2 : 0; }

bool good_tensor(const gs_tensor& t) {
  const size_t es = type_size(t.dtype);
  if (!es || t.rows < 0 || t.cols < 0) return false;
  if (t.rows == 0 || t.cols == 0) return true;
  if (!t.data || !aligned(t.data, es)) return false;
  if (t.rows > 1 && t.row_stride < t.cols) return false;
  return t.cols <= INT64_MAX / 8 / t.rows;
}

bool good_list(const gs_tensor* t, int32_t count) {
  if (count < 0 || (count > 0 && !t)) return false;
  for (int32_t i = 0; i < count; ++i)
    if (!good_tensor(t[i])) return false;
  return true;
}

// Bytes from the first to behind the last element of a tensor.
size_t extent(const gs_tensor& t) {
  if (t.rows == 0 || t.cols == 0) return 0;
  return (size_t)((t.rows - 1) * t.row_stride + t.cols) * type_size(t.dtype);
}

// One piece of contiguous elements?
bool one_piece(const gs_tensor& t) { return t.rows == 1 || t.row_stride == t.cols; }

// Brings a pair to common rows and columns: one piece is cut like the other
// tensor's rows.  False if the pair does not hold the same elements.
bool pair_up(gs_tensor* a, gs_tensor* b) {
  if (a->dtype != b->dtype || a->rows * a->cols != b->rows * b->cols) return false;
  auto recut = [](gs_tensor* t, int64_t rows, int64_t cols) {
    t->rows = rows;
    t->cols = t->row_stride = cols;
  };
  const int64_t size = a->rows * a->cols;
  const bool pa = one_piece(*a), pb = one_piece(*b);
  if (pa) recut(a, pb ? 1 : b->rows, pb ? size : b->cols);
  if (pb) recut(b, a->rows, a->cols);
  return a->rows == b->rows && a->cols == b->cols;
}

// Fills tab with up to kMaxTensors non-empty tensors from *at on.
void fill(Table& tab, const gs_tensor* src, const gs_tensor* dst, int32_t count, int32_t* at) {
  tab.count = 0;
  tab.units = 0;
  for (; *at < count && tab.count < kMaxTensors; ++*at) {
    gs_tensor t = src[*at], d = dst ? dst[*at] : t;
    if (t.rows == 0 || t.cols == 0) continue;
    pair_up(&t, &d);
    Entry& e = tab.t[tab.count++];
    e.src = t.data;
    e.dst = d.data;
    e.dtype = t.dtype;
    e.size = t.rows * t.cols;
    e.cols = t.cols;
    e.src_stride = t.row_stride;
    e.dst_stride = d.row_stride;
    e.unit0 = tab.units;
    tab.units += (e.size + kUnit - 1) / kUnit;
  }
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" size_t gs_grad_norm_workspace_size(int32_t count) {
  if (count < 0) return 0;
  const size_t launches = (size_t)(count + kMaxTensors - 1) / kMaxTensors;
  return round_up((launches ? launches : 1) * kNormBlocks * sizeof(double), 256);
}

extern "C" gs_status gs_grad_norm(const gs_tensor* tensors, int32_t count, double max_norm,
                                  double eps, float* clip, void* ws, size_t ws_bytes,
                                  int32_t* dev_status, gs_stream stream) {
  if (!good_list(tensors, count) || !clip || !aligned(clip, 8)) return GS_ERR_ARG;
  if (!(max_norm >= 0) || !isfinite(max_norm) || !(eps >= 0) || !isfinite(eps)) return GS_ERR_ARG;
  if (!ws || ws_bytes < gs_grad_norm_workspace_size(count)) return GS_ERR_CAPACITY;
  if (!aligned(ws, 256)) return GS_ERR_ARG;
  cudaStream_t s = to_stream(stream);
  double* part = static_cast<double*>(ws);
  int parts = 0;
  static thread_local Table tab;
  for (int32_t at = 0; at < count;) {
    fill(tab, tensors, nullptr, count, &at);
    if (tab.count == 0) break;
    const unsigned blocks = (unsigned)(tab.units < kNormBlocks ? tab.units : kNormBlocks);
    k_sum_squares<<<blocks, kThreads, 0, s>>>(tab, part + parts);
    GS_LAUNCH_CHECK();
    parts += (int)blocks;
  }
  k_clip_coef<<<1, kThreads, 0, s>>>(part, parts, max_norm, eps, clip, dev_status);
  GS_LAUNCH_CHECK();
  return GS_OK;
}

extern "C" gs_status gs_grad_clip(const gs_tensor* src, const gs_tensor* dst, int32_t count,
                                  const float* clip, gs_stream stream) {
  if (!good_list(src, count) || !good_list(dst, count) || !clip || !aligned(clip, 8))
    return GS_ERR_ARG;
  for (int32_t i = 0; i < count; ++i) {
    gs_tensor x = src[i], y = dst[i];
    if (!pair_up(&x, &y)) return GS_ERR_ARG;
    // in place or apart: a copy that overlaps its source is refused
    const char* a = static_cast<const char*>(x.data);
    const char* b = static_cast<const char*>(y.data);
    if (a == b && x.row_stride == y.row_stride) continue;
    if (extent(x) && a < b + extent(y) && b < a + extent(x)) return GS_ERR_ARG;
  }
  cudaStream_t s = to_stream(stream);
  static thread_local Table tab;
  for (int32_t at = 0; at < count;) {
    fill(tab, src, dst, count, &at);
    if (tab.count == 0) break;
    const unsigned blocks = (unsigned)(tab.units < 148 * 16 ? tab.units : 148 * 16);
    k_clip<<<blocks, kThreads, 0, s>>>(tab, clip);
    GS_LAUNCH_CHECK();
  }
  return GS_OK;
}
