// The global gradient norm over many tensors, clipping, and Adam on the
// clipped gradient.
//
//   N = sqrt(sum over all elements of g^2),   c = min(1, max_norm / (N + eps))
//   clipped g = c g,   Adam on c g.
// The norm is a sum over everything before anything can be scaled, so the
// coefficient stays on the device: Adam (or the clipping copy) reads it.
// The tensors' descriptors are passed by value, so that a call can be captured
// into a graph and leaves nothing behind.  Bound by HBM: 59 planes of 6M
// floats (1.4 GB) take 199 us for the norm (7.1 TB/s) and 405 for the clipped
// copy (7.0 TB/s read and written).  32 KB units and many short blocks: 16 KB
// units took 691 us for both against 637, eight blocks per SM 758.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include <memory>
#include <new>

#include "gs_internal.cuh"

namespace gs {
namespace {

constexpr int kThreads = 256;
constexpr int kUnitShift = 15, kUnitBytes = 1 << kUnitShift;  // of a row, that a block takes at a time
constexpr int kFlatUnit = 4096;    // elements, where rows are too short for that
constexpr int kShortRow = 1024;    // columns below which rows are short
constexpr int kMaxTensors = 256;   // tensors per launch, passed by value
constexpr int kFewTensors = 16, kSomeTensors = 64, kManyTensors = 128;  // quicker to pass
constexpr int kNormBlocks = 148 * 32;
constexpr int kClipBlocks = 148 * 64;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// 16 bytes of elements
template <class T>
union Vec {
  uint4 raw;
  T x[16 / sizeof(T)];
  __device__ Vec() {}
};

struct Entry {
  const void* src;
  void* dst;
  int64_t cols, src_stride, dst_stride, size;  // size = rows * cols
  uint32_t unit0;                              // first unit of this tensor
  uint32_t row_units;                          // units per row; 0: rows are short
  int32_t dtype;
};

template <int N>
struct Table {
  uint32_t units;
  int32_t count;
  Entry t[N];
};

constexpr int kVecs = kUnitBytes / 16 / kThreads;  // vectors of a unit per thread

// Unit u of tensor e: a stretch of one row, cut into single elements up to
// the source's first 16-byte boundary, vectors, and the rest.
template <class T>
struct Stretch {
  const T* src;
  T* dst;
  int len, head, nv;
  __device__ Stretch(const Entry& e, int64_t u) {
    constexpr int V = 16 / sizeof(T), kUnit = kUnitBytes / sizeof(T);
    u -= e.unit0;
    const int64_t r = u / e.row_units, c0 = (u - r * e.row_units) * kUnit;
    len = (int)min((int64_t)kUnit, e.cols - c0);
    src = static_cast<const T*>(e.src) + r * e.src_stride + c0;
    dst = static_cast<T*>(e.dst) + r * e.dst_stride + c0;
    head = min(len, (int)(((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / sizeof(T)));
    nv = (len - head) / V;
  }
  // one(i): this thread's single elements before and behind the vectors
  template <class F>
  __device__ __forceinline__ void ends(F&& one) const {
    const int t = threadIdx.x % kThreads, tail = head + nv * (16 / (int)sizeof(T));
    if (t < head) one(t);
    if (t < len - tail) one(tail + t);
  }
};

// Unit u of a tensor with short rows: single elements, with a division each.
template <class T, class F>
__device__ __forceinline__ void short_rows(const Entry& e, int64_t u, F&& one) {
  const int64_t a = (u - e.unit0) * kFlatUnit, b = min(a + kFlatUnit, e.size);
  for (int64_t i = a + threadIdx.x % kThreads; i < b; i += kThreads) {
    const int64_t r = i / e.cols, c = i - r * e.cols;
    one(static_cast<const T*>(e.src) + r * e.src_stride + c,
        static_cast<T*>(e.dst) + r * e.dst_stride + c);
  }
}

// f(tensor, unit) for this block's units, in turn from the first or the last
template <bool BACK, int N, class F>
__device__ __forceinline__ void each_unit(const Table<N>& tab, int64_t first, int64_t step, F&& f) {
  for (int64_t k = first; k < tab.units; k += step) {
    const int64_t u = BACK ? tab.units - 1 - k : k;
    int lo = 0, hi = tab.count - 1;  // the last tensor with unit0 <= u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.t[mid].unit0 <= u) lo = mid;
      else hi = mid - 1;
    }
    f(tab.t[lo], u);
  }
}

// Sum of squares of this thread's elements of the units first, first + step,
// ..., a unit by kThreads threads.  fp64: a square of a finite fp32 value
// neither overflows nor vanishes there, and a sum over 2^40 elements keeps
// 1e-4 of its last fp32 place.
template <int N>
__device__ __forceinline__ double sum_squares(const Table<N>& tab, int64_t first, int64_t step) {
  double sum = 0.0;
  auto unit = [&](auto zero, const Entry& e, int64_t u) {
    using T = decltype(zero);
    constexpr int V = 16 / sizeof(T);
    auto add = [&](float x) { sum = fma((double)x, (double)x, sum); };
    if (e.row_units == 0) return short_rows<T>(e, u, [&](const T* p, T*) { add(to_f(*p)); });
    const Stretch<T> x(e, u);
    Vec<T> buf[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int i = threadIdx.x % kThreads + k * kThreads;
      buf[k].raw = i < x.nv ? __ldg(reinterpret_cast<const uint4*>(x.src + x.head) + i)
                            : make_uint4(0, 0, 0, 0);
    }
    x.ends([&](int i) { add(to_f(x.src[i])); });
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) add(to_f(buf[k].x[i]));
  };
  each_unit<false>(tab, first, step, [&](const Entry& e, int64_t u) {
    if (e.dtype == GS_F32) unit(0.f, e, u);
    else if (e.dtype == GS_F16) unit(__half(), e, u);
    else unit(__nv_bfloat16(), e, u);
  });
  return sum;
}

// Sum over the block, valid in thread 0.
template <int WARPS>
__device__ __forceinline__ double block_sum(double sum, double* s_warp) {
  sum = warp_sum(sum);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < WARPS; ++w) sum += s_warp[w];
  return sum;
}

struct CoefArgs {
  double max_norm, eps;
  float* clip;
  int32_t* dev_status;
};

// clip[0] = norm, clip[1] = coefficient (see gs.h for non-finite norms)
__device__ __forceinline__ void write_clip(double sum, const CoefArgs& a) {
  const double norm = sqrt(sum);
  const double c = a.max_norm / (norm + a.eps);
  a.clip[0] = (float)norm;
  a.clip[1] = (float)(c < 1.0 ? c : isnan(norm) ? norm : 1.0);
  if (!isfinite(norm)) dev_flag(a.dev_status, GS_DEV_NONFINITE);
}

template <int N>
__global__ void __launch_bounds__(kThreads)
k_sum_squares(const __grid_constant__ Table<N> tab, double* __restrict__ part) {
  __shared__ double s_warp[kThreads / 32];
  wait_for_prior_grids();
  const double sum = block_sum<kThreads / 32>(sum_squares(tab, blockIdx.x, gridDim.x), s_warp);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads)
k_clip_coef(const double* __restrict__ part, int n, const CoefArgs a) {
  __shared__ double s_warp[kThreads / 32];
  wait_for_prior_grids();
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) sum += part[i];
  sum = block_sum<kThreads / 32>(sum, s_warp);
  if (threadIdx.x == 0) write_clip(sum, a);
}

// Up to kClusterUnits units in one launch: a cluster of 8 blocks, four units
// in each; the blocks' sums meet in the first one's shared memory.  A launch
// less is 1.2 us of host time (five small tensors: 12.5 us for norm and clip
// against 13.8); in a graph one unit takes 2.4 us against 2.8 in two launches,
// 30 units 3.8 against 2.7.
constexpr int kCluster = 8, kClusterThreads = 1024;
constexpr uint32_t kClusterUnits = kCluster * kClusterThreads / kThreads;
template <int N>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kClusterThreads)
k_norm_cluster(const __grid_constant__ Table<N> tab, const CoefArgs a) {
  constexpr int G = kClusterThreads / kThreads;
  __shared__ double s_warp[kClusterThreads / 32];
  __shared__ double s_block[kCluster];
  // every block has started before one writes to another's shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  wait_for_prior_grids();
  const double sum = block_sum<kClusterThreads / 32>(
      sum_squares(tab, blockIdx.x * G + threadIdx.x / kThreads, kCluster * G), s_warp);
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (threadIdx.x == 0) {
    unsigned to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_addr(&s_block[blockIdx.x])));
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(sum) : "memory");
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    double all = 0.0;
    for (int k = 0; k < kCluster; ++k) all += s_block[k];
    write_clip(all, a);
  }
}

// The units are taken from the last to the first: what the norm read last is
// still in L2.
template <int N>
__global__ void __launch_bounds__(kThreads)
k_clip(const __grid_constant__ Table<N> tab, const float* __restrict__ clip) {
  wait_for_prior_grids();
  const float c = clip[1];
  auto unit = [&](auto zero, const Entry& e, int64_t u) {
    using T = decltype(zero);
    constexpr int V = 16 / sizeof(T);
    if (e.row_units == 0)
      return short_rows<T>(e, u, [&](const T* p, T* q) { put(q, clipped(c, to_f(*p))); });
    const Stretch<T> x(e, u);
    const bool aligned_dst = (reinterpret_cast<uintptr_t>(x.dst + x.head) & 15) == 0;
    Vec<T> buf[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int i = threadIdx.x + k * kThreads;
      if (i < x.nv) buf[k].raw = __ldcs(reinterpret_cast<const uint4*>(x.src + x.head) + i);
    }
    x.ends([&](int i) { put(x.dst + i, clipped(c, to_f(x.src[i]))); });
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int i = threadIdx.x + k * kThreads;
      if (i >= x.nv) break;
      Vec<T> w;
#pragma unroll
      for (int j = 0; j < V; ++j) put(&w.x[j], clipped(c, to_f(buf[k].x[j])));
      if (aligned_dst) {
        __stcs(reinterpret_cast<uint4*>(x.dst + x.head) + i, w.raw);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) x.dst[x.head + i * V + j] = w.x[j];
      }
    }
  };
  each_unit<true>(tab, blockIdx.x, gridDim.x, [&](const Entry& e, int64_t u) {
    if (c == 1.0f && e.src == e.dst) return;  // in place and nothing to clip
    if (e.dtype == GS_F32) unit(0.f, e, u);
    else if (e.dtype == GS_F16) unit(__half(), e, u);
    else unit(__nv_bfloat16(), e, u);
  });
}

size_t type_size(int dtype) { return dtype == GS_F32 ? 4 : dtype == GS_F16 || dtype == GS_BF16 ? 2 : 0; }

bool good_tensor(const gs_tensor& t) {
  const size_t es = type_size(t.dtype);
  if (!es || t.rows < 0 || t.cols < 0) return false;
  if (t.rows == 0 || t.cols == 0) return true;
  if (!t.data || !aligned(t.data, es)) return false;
  if (t.rows > 1 && t.row_stride < t.cols) return false;
  int64_t bytes;
  return !__builtin_mul_overflow(t.cols, t.rows, &bytes) && bytes <= INT64_MAX / 8;
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

// The addresses where a list's tensors start, kept by hashing: finds a tensor
// that is written twice, or read as one entry and written as another.  Their
// blocks would race, and a tensor listed twice would be scaled once or twice.
class Starts {
 public:
  // `slots`: a power of two above the number of entries, all 0
  Starts(uintptr_t* slots, size_t size) : slots_(slots), mask_(size - 1) {}
  // false if it starts where another entry does, and one of the two is written
  bool add(const void* p, bool written) {
    const uintptr_t key = reinterpret_cast<uintptr_t>(p);  // even: two bytes an element at least
    size_t i = (key * 0x9e3779b97f4a7c15ull) >> 32;        // 2^64 / golden ratio
    for (;; ++i) {
      uintptr_t& slot = slots_[i & mask_];
      if (slot == 0) {
        slot = key | (uintptr_t)written;
        return true;
      }
      if ((slot & ~(uintptr_t)1) == key && (written || (slot & 1))) return false;
    }
  }

 private:
  uintptr_t* slots_;
  size_t mask_;
};

// Fills tab with up to N non-empty tensors from *at on; false if
// 32 bits do not count their units.
template <int N>
bool fill(Table<N>& tab, const gs_tensor* src, const gs_tensor* dst, int32_t count, int32_t* at) {
  tab.count = 0;
  int64_t units = 0;
  for (; *at < count && tab.count < N; ++*at) {
    gs_tensor t = src[*at], d = t;
    if (t.rows == 0 || t.cols == 0) continue;
    if (dst) {
      d = dst[*at];
      pair_up(&t, &d);
    } else if (one_piece(t)) {
      t.cols *= t.rows;
      t.rows = 1;
    }
    Entry& e = tab.t[tab.count++];
    e.src = t.data;
    e.dst = d.data;
    e.dtype = t.dtype;
    e.size = t.rows * t.cols;
    e.cols = t.cols;
    e.src_stride = t.row_stride;
    e.dst_stride = d.row_stride;
    e.unit0 = (uint32_t)units;
    const int shift = t.dtype == GS_F32 ? kUnitShift - 2 : kUnitShift - 1;  // elements per unit
    const int64_t row_units = ((t.cols - 1) >> shift) + 1;
    const bool is_short = t.rows > 1 && t.cols < kShortRow;
    e.row_units = is_short ? 0 : (uint32_t)row_units;
    units += is_short ? (e.size + kFlatUnit - 1) / kFlatUnit : t.rows * row_units;
    if (units > (int64_t)UINT32_MAX) return false;
  }
  tab.units = (uint32_t)units;
  return true;
}

template <int N>
gs_status norm_impl(const gs_tensor* tensors, int32_t count, double* part, const CoefArgs& a,
                    cudaStream_t s) {
  Table<N> tab;
  int parts = 0;
  for (int32_t at = 0; at < count;) {
    if (!fill(tab, tensors, nullptr, count, &at)) return GS_ERR_UNSUPPORTED;
    if (tab.units <= kClusterUnits && at == count && parts == 0) {
      GS_TRY(launch_dependent(k_norm_cluster<N>, kCluster, kClusterThreads, 0, s, tab, a));
      GS_LAUNCH_CHECK();
      return GS_OK;
    }
    if (tab.count == 0) break;
    const unsigned blocks = (unsigned)(tab.units < kNormBlocks ? tab.units : kNormBlocks);
    GS_TRY(launch_dependent(k_sum_squares<N>, blocks, kThreads, 0, s, tab, part + parts));
    GS_LAUNCH_CHECK();
    parts += (int)blocks;
  }
  GS_TRY(launch_dependent(k_clip_coef, 1, kThreads, 0, s, part, parts, a));
  GS_LAUNCH_CHECK();
  return GS_OK;
}

template <int N>
gs_status clip_impl(const gs_tensor* src, const gs_tensor* dst, int32_t count, const float* clip,
                    cudaStream_t s) {
  Table<N> tab;
  for (int32_t at = 0; at < count;) {
    if (!fill(tab, src, dst, count, &at)) return GS_ERR_UNSUPPORTED;
    if (tab.count == 0) break;
    const unsigned blocks = (unsigned)(tab.units < kClipBlocks ? tab.units : kClipBlocks);
    GS_TRY(launch_dependent(k_clip<N>, blocks, kThreads, 0, s, tab, clip));
    GS_LAUNCH_CHECK();
  }
  return GS_OK;
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
  const CoefArgs a{max_norm, eps, clip, dev_status};
  double* part = static_cast<double*>(ws);
  cudaStream_t s = to_stream(stream);
  if (count <= kFewTensors) return norm_impl<kFewTensors>(tensors, count, part, a, s);
  if (count <= kSomeTensors) return norm_impl<kSomeTensors>(tensors, count, part, a, s);
  if (count <= kManyTensors) return norm_impl<kManyTensors>(tensors, count, part, a, s);
  return norm_impl<kMaxTensors>(tensors, count, part, a, s);
}

extern "C" gs_status gs_grad_clip(const gs_tensor* src, const gs_tensor* dst, int32_t count,
                                  const float* clip, gs_stream stream) {
  if (!good_list(src, count) || !good_list(dst, count) || !clip || !aligned(clip, 8))
    return GS_ERR_ARG;
  uintptr_t few[4 * kMaxTensors];
  std::unique_ptr<uintptr_t[]> many;
  size_t slots = 4 * kFewTensors;
  while (slots < 4 * (size_t)count) slots *= 2;
  if (count > kMaxTensors) {
    many.reset(new (std::nothrow) uintptr_t[slots]);
    if (!many) return GS_ERR_CAPACITY;
  }
  uintptr_t* table = many ? many.get() : few;
  memset(table, 0, slots * sizeof(uintptr_t));
  Starts starts(table, slots);
  for (int32_t i = 0; i < count; ++i) {
    gs_tensor x = src[i], y = dst[i];
    if (!pair_up(&x, &y)) return GS_ERR_ARG;
    if (extent(x) == 0) continue;
    // in place or apart: a copy that overlaps its source is refused
    const char* a = static_cast<const char*>(x.data);
    const char* b = static_cast<const char*>(y.data);
    if (!starts.add(b, true)) return GS_ERR_ARG;
    if (a == b && x.row_stride == y.row_stride) continue;
    if (a < b + extent(y) && b < a + extent(x)) return GS_ERR_ARG;
    if (!starts.add(a, false)) return GS_ERR_ARG;
  }
  cudaStream_t s = to_stream(stream);
  if (count <= kFewTensors) return clip_impl<kFewTensors>(src, dst, count, clip, s);
  if (count <= kSomeTensors) return clip_impl<kSomeTensors>(src, dst, count, clip, s);
  if (count <= kManyTensors) return clip_impl<kManyTensors>(src, dst, count, clip, s);
  return clip_impl<kMaxTensors>(src, dst, count, clip, s);
}
