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

// V elements of the table's type as one load of V * sizeof(T) bytes
template <class T, int V>
struct alignas(sizeof(T) * V) Pack {
  T x[V];
};

// Division by a number fixed at launch, for dividends below 2^31:
// q = (x * m) >> 32 >> s with m = ceil(2^(32+s) / d), s = ceil(log2 d) - 1
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994); d = 1 is left out by the caller's `one`.
struct Div {
  uint32_t d, m, s;
  __host__ explicit Div(uint32_t dd) : d(dd), m(0), s(0) {
    if (d <= 1) return;
    while ((2ull << s) < d) ++s;
    m = (uint32_t)(((1ull << (32 + s)) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t quot(uint32_t x) const {
    return d == 1 ? x : __umulhi(x, m) >> s;
  }
};

// out in rows: one thread per V columns of an item, kRowIlp items' vectors in
// flight.  A block takes kThreads * kRowIlp consecutive vectors.
constexpr int kRowIlp = 4;
template <class TT, class TO, int V>
__global__ void __launch_bounds__(kThreads)
k_lookup_rows(const TT* __restrict__ table, int64_t ld, int64_t rows,
              const int32_t* __restrict__ ids, int64_t n_ids, const int32_t* __restrict__ index,
              float scale, TO* __restrict__ out, int64_t n, int64_t rs, Div nv, int items,
              int32_t* dev_status) {
  const int64_t j0 = (int64_t)blockIdx.x * items;  // items per block
  const uint32_t total = (uint32_t)min((int64_t)items, n - j0) * nv.d;
  for (uint32_t e0 = threadIdx.x; e0 < total; e0 += kThreads * kRowIlp) {
    Pack<TT, V> in[kRowIlp];
    uint32_t at[kRowIlp], c[kRowIlp];
    bool has[kRowIlp];
#pragma unroll
    for (int k = 0; k < kRowIlp; ++k) {
      const uint32_t e = min(e0 + k * kThreads, total - 1);
      at[k] = nv.quot(e);
      c[k] = (e - at[k] * nv.d) * V;
      const int32_t id = id_of(ids, n_ids, index, j0 + at[k], rows, dev_status);
      has[k] = id >= 0;
      if (has[k])
        in[k] = *reinterpret_cast<const Pack<TT, V>*>(table + (int64_t)id * ld + c[k]);
    }
#pragma unroll
    for (int k = 0; k < kRowIlp; ++k) {
      if (e0 + k * kThreads >= total) break;
      Pack<TO, V> w;
#pragma unroll
      for (int i = 0; i < V; ++i) w.x[i] = from_f<TO>(has[k] ? scale * to_f(in[k].x[i]) : 0.f);
      *reinterpret_cast<Pack<TO, V>*>(out + (j0 + at[k]) * rs + c[k]) = w;
    }
  }
}

// out in planes: one thread per item.  It loads up to NW 32-bit words of its
// row (a share of the columns) into registers in 16-byte vectors, all in
// flight at once, and the warp writes 32 neighbouring items of a plane with
// each store: no shared memory, no barrier.
//
// Rows that do not start on 16 bytes are covered by the aligned vectors that
// they touch and moved into place by selects (by 2 words, by 1, by half a
// word).  Vectors that reach over the table's first or last byte are read by
// element.
template <class TT>
__device__ __forceinline__ uint4 load_cover(uintptr_t p, uintptr_t first, uintptr_t last) {
  if (p >= first && p + 16 <= last) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(TT)); ++i) {
    const uintptr_t q = p + i * sizeof(TT);
    if (q < first || q >= last) continue;
    if (sizeof(TT) == 4) w[i] = *reinterpret_cast<const uint32_t*>(q);
    else w[i / 2] |= (uint32_t) * reinterpret_cast<const uint16_t*>(q) << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <class TT>
__device__ __forceinline__ float element(const uint32_t* w, int c);
template <>
__device__ __forceinline__ float element<float>(const uint32_t* w, int c) {
  return __uint_as_float(w[c]);
}
template <>
__device__ __forceinline__ float element<__half>(const uint32_t* w, int c) {
  return __half2float(__ushort_as_half((unsigned short)(w[c / 2] >> (16 * (c & 1)))));
}
template <>
__device__ __forceinline__ float element<__nv_bfloat16>(const uint32_t* w, int c) {
  return __uint_as_float(c & 1 ? w[c / 2] & 0xffff0000u : w[c / 2] << 16);
}

// 32 bytes as one load (one whole sector of L2 and L1)
__device__ __forceinline__ void load_32(uint32_t* w, const void* p) {
  asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
      : "l"(p));
}

// NW words of a row from column c0 on (`width` of its columns if !FULL)
template <class TT, int NW, int ALIGNED, bool FULL>
__device__ __forceinline__ void load_words(uint32_t* w, const TT* table, int64_t ld, int64_t rows,
                                           int table_cols, int64_t id, int c0, int width) {
  constexpr int E = 4 / sizeof(TT), NL = ALIGNED ? NW : NW + 4;
  const uintptr_t first = reinterpret_cast<uintptr_t>(table);
  const uintptr_t row = first + (uintptr_t)(id * ld + c0) * sizeof(TT);
  if (ALIGNED == 32) {
#pragma unroll
    for (int v = 0; v < NW / 8; ++v)
      if (FULL || v * 8 * E < width) load_32(w + 8 * v, reinterpret_cast<const uint4*>(row) + 2 * v);
  } else if (ALIGNED == 16) {
#pragma unroll
    for (int v = 0; v < NW / 4; ++v)
      if (FULL || v * 4 * E < width)
        *reinterpret_cast<uint4*>(w + 4 * v) = __ldg(reinterpret_cast<const uint4*>(row) + v);
  } else {
    const uintptr_t last = first + (uintptr_t)((rows - 1) * ld + table_cols) * sizeof(TT);
    const uintptr_t p = row & ~(uintptr_t)15, end = row + (uintptr_t)width * sizeof(TT);
#pragma unroll
    for (int v = 0; v < NL / 4; ++v)
      if (p + 16 * v < end)
        *reinterpret_cast<uint4*>(w + 4 * v) = load_cover<TT>(p + 16 * v, first, last);
    const unsigned o = (unsigned)(row & 15);
#pragma unroll
    for (int k = 0; k + 2 < NL; ++k) w[k] = o & 8 ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k + 3 < NL; ++k) w[k] = o & 4 ? w[k + 1] : w[k];
    if (E == 2) {
      const unsigned sh = (o & 2) * 8;
#pragma unroll
      for (int k = 0; k + 4 < NL; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], sh);
    }
  }
}

template <class TT, class TO, int NW, int ALIGNED>
__global__ void __launch_bounds__(kThreads, NW > 16 ? 3 : 5)
k_lookup_planes(const TT* __restrict__ table, int64_t ld, int64_t rows, int table_cols,
                const int32_t* __restrict__ ids, int64_t n_ids, const int32_t* __restrict__ index,
                float scale, TO* __restrict__ out, int64_t n, int64_t cs, int32_t* dev_status) {
  constexpr int C = NW * 4 / sizeof(TT);           // columns at a time
  constexpr int NL = ALIGNED ? NW : NW + 4;        // words loaded
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= n) return;
  const int32_t id = id_of(ids, n_ids, index, j, rows, dev_status);
  const bool has = id >= 0;
  TO* o = out + j;
  uint32_t w[NL];
  const auto store = [&](int c) {
    *o = from_f<TO>(has ? scale * element<TT>(w, c) : 0.f);
    o += cs;
    asm volatile("" : "+l"(o));  // one running pointer, not C addresses in registers
  };
  int c0 = 0;
  for (; c0 + C <= table_cols; c0 += C) {
    load_words<TT, NW, ALIGNED, true>(w, table, ld, rows, table_cols, has ? id : 0, c0, C);
#pragma unroll
    for (int c = 0; c < C; ++c) store(c);
  }
  if (c0 < table_cols) {
    const int width = table_cols - c0;
    load_words<TT, NW, ALIGNED, false>(w, table, ld, rows, table_cols, has ? id : 0, c0, width);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c < width) store(c);
  }
}

// out in planes, rows of more than 32 bytes on 16-byte boundaries: a warp
// fetches the rows of 32 items together (lanes along the row, so that a line
// is one request; a lane that reads its own row makes one request for every
// 32 bytes, which bounded the kernel above: 309 us against this one's at
// 6M x 48) by asynchronous copies into its own part of shared memory, and
// each lane then reads its item's row from there, 16 bytes at a time.  The
// row pitch of 4 words more than a multiple of 16 keeps those reads free of
// bank conflicts.  Many short blocks hide the latencies; persistent blocks
// that fetch the next ids ahead took 293 us, these take 286.
constexpr int kStageWarps = 4, kStageVecs = 12;            // 192 bytes of a row at a time
constexpr int kStagePitch = 4 * kStageVecs + 4;            // words

__device__ __forceinline__ void copy_16_async(void* smem, const void* p, bool has) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(smem)), "l"(p),
               "r"(has ? 16 : 0)
               : "memory");
}

template <class TT, class TO>
__global__ void __launch_bounds__(32 * kStageWarps)
k_lookup_planes_staged(const TT* __restrict__ table, int64_t ld, int64_t rows, int cols,
                       const int32_t* __restrict__ ids, int64_t n_ids,
                       const int32_t* __restrict__ index, float scale, TO* __restrict__ out,
                       int64_t n, int64_t cs, int32_t* dev_status) {
  constexpr int V = 16 / sizeof(TT);
  __shared__ __align__(16) uint32_t s_rows[kStageWarps][32 * kStagePitch];
  const int lane = threadIdx.x & 31;
  uint32_t* s = s_rows[threadIdx.x >> 5];
  const int64_t j = ((int64_t)blockIdx.x * kStageWarps + (threadIdx.x >> 5)) * 32 + lane;
  const int32_t id = j < n ? id_of(ids, n_ids, index, j, rows, dev_status) : -1;
  for (int c0 = 0; c0 < cols; c0 += kStageVecs * V) {
    const int nv = min(kStageVecs, (cols - c0) / V);
    int r = lane / nv, v = lane - r * nv;
    const int dr = 32 / nv, dv = 32 - dr * nv;
    for (int k = 0; k < nv; ++k) {
      const int32_t row = __shfl_sync(0xffffffffu, id, r);
      copy_16_async(s + r * kStagePitch + 4 * v,
                    table + (int64_t)(row < 0 ? 0 : row) * ld + c0 + v * V, row >= 0);
      r += dr;
      v += dv;
      if (v >= nv) {
        v -= nv;
        ++r;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    if (j < n) {
      TO* o = out + (int64_t)c0 * cs + j;
      for (int q = 0; q < nv; ++q) {
        uint32_t w[4];
        *reinterpret_cast<uint4*>(w) =
            *reinterpret_cast<const uint4*>(s + lane * kStagePitch + 4 * q);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          *o = from_f<TO>(id >= 0 ? scale * element<TT>(w, i) : 0.f);
          o += cs;
        }
      }
    }
    __syncwarp();
  }
}

// Sort keys and values of the gradient's items: key = id, value = j.  An
// item without a row takes the last key and a negative value, which adds
// nothing, so that the keys need no bit more than the rows do.
__global__ void __launch_bounds__(kThreads)
k_lookup_keys(const int32_t* __restrict__ ids, int64_t n_ids, const int32_t* __restrict__ index,
              int64_t n, int64_t rows, uint32_t* __restrict__ keys, int32_t* __restrict__ vals,
              int32_t* dev_status) {
  wait_for_prior_grids();
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= n) return;
  const int32_t id = id_of(ids, n_ids, index, j, rows, dev_status);
  keys[j] = id >= 0 ? (uint32_t)id : (uint32_t)(rows - 1);
  vals[j] = id >= 0 ? (int32_t)j : -1;
}

// Planes to rows (pitch `vecs` 16-byte vectors, columns past the last one
// unset): the sums below read whole rows in the order of their ids, and a row
// in planes costs a 32-byte sector for every element.  A warp turns 32 items
// in its own part of shared memory; the rows leave as one contiguous piece.
template <class T>
__global__ void __launch_bounds__(32 * kStageWarps)
k_planes_to_rows(const T* __restrict__ g, int64_t cs, int cols, int64_t n, uint4* __restrict__ out,
                 int vecs) {
  constexpr int V = 16 / sizeof(T);
  __shared__ __align__(16) uint32_t s_rows[kStageWarps][32 * kStagePitch];
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31;
  uint32_t* s = s_rows[threadIdx.x >> 5];
  const int64_t j0 = ((int64_t)blockIdx.x * kStageWarps + (threadIdx.x >> 5)) * 32, j = j0 + lane;
  if (j0 >= n) return;
  const int items = (int)min((int64_t)32, n - j0);
  for (int v0 = 0; v0 < vecs; v0 += kStageVecs) {
    const int nv = min(kStageVecs, vecs - v0);
    if (j < n) {
      const T* p = g + (int64_t)v0 * V * cs + j;
#pragma unroll 4
      for (int q = 0; q < nv; ++q) {
        union {
          uint4 raw;
          uint32_t w[4];
        } x;
        x.raw = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if ((v0 + q) * V + i < cols) {
            if (sizeof(T) == 4) x.w[i] = __ldcs(reinterpret_cast<const uint32_t*>(p));
            else x.w[i / 2] |= (uint32_t)__ldcs(reinterpret_cast<const uint16_t*>(p)) << (16 * (i & 1));
          }
          p += cs;
        }
        *reinterpret_cast<uint4*>(s + lane * kStagePitch + 4 * q) = x.raw;
      }
    }
    __syncwarp();
    int r = lane / nv, v = lane - r * nv;
    const int dr = 32 / nv, dv = 32 - dr * nv;
    for (int k = 0; k < nv; ++k) {
      if (r < items)
        out[(j0 + r) * vecs + v0 + v] = *reinterpret_cast<const uint4*>(s + r * kStagePitch + 4 * v);
      r += dr;
      v += dv;
      if (v >= nv) {
        v -= nv;
        ++r;
      }
    }
    __syncwarp();
  }
}

// Sums of runs of equal keys over a list of n entries, entry r standing for
// the row order[r] of g (or row r).  The list is cut into chunks of R
// entries; a thread sums V columns of one chunk in order, the loads of kRunIlp
// entries in flight.  A run that lies inside a chunk goes to dtable.  What a
// chunk holds of a run that goes on across its border is a partial: entry
// 2 chunk for a run that came in from the chunk before, 2 chunk + 1 for one
// that starts here and goes on.  A chunk inside one run writes its sum at
// 2 chunk and zeros at 2 chunk + 1, so that the partials of one run are
// neighbours; unused partials have the key kNoRow.  The partials are summed
// by the same kernel.  keys and order are readable up to a multiple of
// kRunIlp entries.
constexpr int kRunIlp = 8;

template <class T, int V>
__global__ void __launch_bounds__(kThreads)
k_run_sums(const uint32_t* __restrict__ keys, const int32_t* __restrict__ order, int64_t n, int R,
           const T* __restrict__ g, int64_t rs, int cols, Div nv, float scale,
           float* __restrict__ dtable, int64_t ld, bool accumulate, uint32_t* __restrict__ pkey,
           float* __restrict__ psum, int ldp) {
  wait_for_prior_grids();
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t chunk = e / nv.d;
  const int c = (int)(e - chunk * nv.d) * V;
  const int64_t a = chunk * R;
  if (a >= n) return;
  const int64_t b = min(a + R, n);
  uint32_t k = keys[a];
  bool head = a > 0 && keys[a - 1] == k;  // the run came in from the chunk before
  bool used0 = false, used1 = false;
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.f;
  auto partial = [&](int at, bool zero) {
    const int64_t p = 2 * chunk + at;
    if (c == 0) pkey[p] = k;
#pragma unroll
    for (int i = 0; i < V; ++i) psum[p * ldp + c + i] = zero ? 0.f : sum[i];
    (at ? used1 : used0) = true;
  };
  auto done = [&](bool tail) {
    if (k == kNoRow) return;
    if (head || tail) {
      partial(head ? 0 : 1, false);
      if (head && tail) partial(1, true);
    } else {
      float* d = dtable + (int64_t)k * ld + c;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (V == 1 || c + i < cols) d[i] = accumulate ? d[i] + scale * sum[i] : scale * sum[i];
    }
  };
  for (int64_t r = a; r < b; r += kRunIlp) {
    uint32_t kr[kRunIlp];
    int32_t j[kRunIlp];
#pragma unroll
    for (int q = 0; q < kRunIlp; q += 4) {
      const uint4 kk = *reinterpret_cast<const uint4*>(keys + r + q);
      kr[q] = kk.x, kr[q + 1] = kk.y, kr[q + 2] = kk.z, kr[q + 3] = kk.w;
      if (order) {
        const int4 o = *reinterpret_cast<const int4*>(order + r + q);
        j[q] = o.x, j[q + 1] = o.y, j[q + 2] = o.z, j[q + 3] = o.w;
      }
    }
    Pack<T, V> x[kRunIlp];
#pragma unroll
    for (int q = 0; q < kRunIlp; ++q) {
      if (!order) j[q] = kr[q] == kNoRow ? -1 : 0;
      if (r + q >= b) j[q] = -1;
      if (j[q] >= 0)
        x[q] = *reinterpret_cast<const Pack<T, V>*>(g + (order ? (int64_t)j[q] : r + q) * rs + c);
    }
#pragma unroll
    for (int q = 0; q < kRunIlp; ++q) {
      if (r + q >= b) break;
      if (kr[q] != k) {
        done(false);
        k = kr[q];
        head = false;
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = 0.f;
      }
      if (j[q] >= 0)
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += to_f(x[q].x[i]);
    }
  }
  done(b < n && keys[b] == k);
  if (c == 0) {
    if (!used0) pkey[2 * chunk] = kNoRow;
    if (!used1) pkey[2 * chunk + 1] = kNoRow;
  }
}

// Up to kSmallItems items, in one launch: a block owns a range of the table's
// rows.  It picks the items with ids in its range (in order), sorts them by id
// in shared memory (the rank of an item is the number of items before it),
// sums the runs of equal ids with teams of threads, each a stretch of the
// sorted list, joins the teams' partial runs in order, and clears the rows
// that nothing used.  Every block reads all ids.
constexpr int kSmallItems = 2048, kSmallPer = kSmallItems / kThreads;
constexpr int kSmallTeams = 64;

template <class T, int V>
__global__ void __launch_bounds__(kThreads)
k_small_grad(const T* __restrict__ g, int64_t rs, int64_t cs, int cols,
             const int32_t* __restrict__ ids, int64_t n_ids, const int32_t* __restrict__ index, int n,
             float scale, float* __restrict__ dtable, int64_t ld, int64_t rows, int64_t per,
             bool accumulate, int32_t* dev_status) {
  __shared__ int32_t s_key[kSmallItems];
  __shared__ uint16_t s_item[kSmallItems];
  __shared__ int s_scan[kThreads / 32 + 1];
  __shared__ int32_t s_pk[2 * kSmallTeams];
  __shared__ float s_part[2 * kThreads * V];
  wait_for_prior_grids();
  const int t = threadIdx.x;
  const int64_t k0 = blockIdx.x * per, k1 = min(k0 + per, rows);
  int32_t key[kSmallPer];
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kSmallPer; ++i) {
    const int j = t * kSmallPer + i;
    const int32_t id = j < n ? id_of(ids, n_ids, index, j, rows, dev_status) : -1;
    key[i] = id >= k0 && id < k1 ? (int32_t)(id - k0) : -1;
    mine += key[i] >= 0;
  }
  if (!accumulate) {
    float* d = dtable + k0 * ld;
    if (ld == cols) {
      const int64_t total = (k1 - k0) * cols;
      for (int64_t i = t; i < total; i += kThreads) d[i] = 0.f;
    } else {
      for (int64_t k = k0; k < k1; ++k, d += ld)
        for (int c = t; c < cols; c += kThreads) d[c] = 0.f;
    }
  }
  int m;
  int at = block_exclusive_scan<int, kThreads / 32>(mine, s_scan, &m);
  if (m == 0) return;
#pragma unroll
  for (int i = 0; i < kSmallPer; ++i)
    if (key[i] >= 0) {
      s_key[at] = key[i];
      s_item[at++] = (uint16_t)(t * kSmallPer + i);
    }
  __syncthreads();  // also: the zeros above are ordered before the sums below
  if (k1 - k0 > 1) {
    int32_t mk[kSmallPer];
    uint16_t mi[kSmallPer];
    int rank[kSmallPer];
#pragma unroll
    for (int i = 0; i < kSmallPer; ++i) {
      const int e = t + i * kThreads;
      if (e < m) {
        mk[i] = s_key[e];
        mi[i] = s_item[e];
        rank[i] = 0;
        for (int f = 0; f < m; ++f) {
          const int32_t kf = s_key[f];
          rank[i] += kf < mk[i] || (kf == mk[i] && f < e);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSmallPer; ++i)
      if (t + i * kThreads < m) {
        s_key[rank[i]] = mk[i];
        s_item[rank[i]] = mi[i];
      }
    __syncthreads();
  }
  const int nv = (cols + V - 1) / V;
  int teams = nv < kThreads ? kThreads / nv : 1;
  teams = min(teams, min(kSmallTeams, (m + 3) / 4));
  const int len = (m + teams - 1) / teams;
  const int width = nv < kThreads ? nv : kThreads;  // vectors of a row at a time
  const int team = t / width, tv = t - team * width;
  for (int v0 = 0; v0 < nv; v0 += width) {
    const int c = (v0 + tv) * V;
    const bool on = team < teams && c < cols;
    const int a = team * len, b = min(a + len, m);
    if (on && tv == 0) s_pk[2 * team] = s_pk[2 * team + 1] = -1;
    if (on && a < b) {
      float sum[V];
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = 0.f;
      int k = s_key[a];
      bool head = a > 0 && s_key[a - 1] == k;
      auto done = [&](bool tail) {
        if (head || tail) {
          const int p = 2 * team + (head ? 0 : 1);
          if (tv == 0) s_pk[p] = k;
#pragma unroll
          for (int i = 0; i < V; ++i) s_part[(p * width + tv) * V + i] = sum[i];
        } else {
          float* d = dtable + (k0 + k) * ld + c;
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (V == 1 || c + i < cols) d[i] = accumulate ? d[i] + scale * sum[i] : scale * sum[i];
        }
      };
      for (int r = a; r < b; r += 4) {
        Pack<T, V> x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (r + q < b) {
            const T* p = g + (int64_t)s_item[r + q] * rs + (int64_t)c * cs;
            if (V > 1) x[q] = *reinterpret_cast<const Pack<T, V>*>(p);
            else x[q].x[0] = *p;
          }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (r + q < b) {
            const int kr = s_key[r + q];
            if (kr != k) {
              done(false);
              k = kr;
              head = false;
#pragma unroll
              for (int i = 0; i < V; ++i) sum[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] += to_f(x[q].x[i]);
          }
      }
      done(b < m && s_key[b] == k);
    }
    __syncthreads();
    // partial runs, joined in order by the first team
    if (team == 0 && c < cols) {
      float sum[V];
      int k = -1;
      auto done = [&]() {
        if (k < 0) return;
        float* d = dtable + (k0 + k) * ld + c;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (V == 1 || c + i < cols) d[i] = accumulate ? d[i] + scale * sum[i] : scale * sum[i];
      };
      for (int p = 0; p < 2 * teams; ++p) {
        const int kp = s_pk[p];
        if (kp < 0) continue;
        if (kp != k) {
          done();
          k = kp;
#pragma unroll
          for (int i = 0; i < V; ++i) sum[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += s_part[(p * width + tv) * V + i];
      }
      done();
    }
    __syncthreads();
  }
}

unsigned blocks_for(int64_t threads) { return (unsigned)((threads + kThreads - 1) / kThreads); }

int key_bits(int64_t rows) { return rows > 1 ? 64 - __builtin_clzll((unsigned long long)(rows - 1)) : 0; }

constexpr int kPartChunk = 64;  // entries per chunk of partials

// Entries per chunk of the items: enough chunks to fill the device, and few
// enough partials that they cost little.
int chunk_of(int64_t n, int nv) {
  const int64_t fill = n * nv / (148 * 1024);
  int R = kRunIlp;
  while (R < 128 && R < fill) R *= 2;
  return R;
}

struct LookupWs {
  uint32_t* keys;
  int32_t* order;
  void* sort;
  size_t sort_bytes;
  uint32_t* pkey[2];
  float* psum[2];
  uint4* rows;  // the items' rows, for a gradient in planes
  int ldp;
  size_t bytes;
};

LookupWs carve_lookup(void* ws, size_t cap, int64_t n, int64_t rows, int cols, int planes_es) {
  LookupWs w{};
  if (n <= kSmallItems) return w;
  Carver cv(ws, cap);
  w.ldp = (cols + 7) / 8 * 8;
  w.keys = cv.take<uint32_t>(round_up(n, kRunIlp));
  w.order = cv.take<int32_t>(round_up(n, kRunIlp));
  w.sort_bytes = gs_sort_workspace_size(n, 4, 0, key_bits(rows));
  w.sort = cv.take<char>(w.sort_bytes);
  const int R = chunk_of(n, (cols + 7) / 8);  // the smallest that any type takes
  int64_t m = 2 * ((n + R - 1) / R);
  for (int k = 0; k < 2; ++k) {
    w.pkey[k] = cv.take<uint32_t>(round_up(m, kRunIlp));
    w.psum[k] = cv.take<float>((size_t)m * w.ldp);
    m = 2 * ((m + kPartChunk - 1) / kPartChunk);
  }
  if (planes_es) w.rows = cv.take<uint4>((size_t)n * ((cols * planes_es + 15) / 16));
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

gs_status plan_lookup(const int32_t* ids, int64_t n_ids, const int32_t* index, int64_t n,
                      int64_t rows, const LookupWs& w, int32_t* dev_status, cudaStream_t s) {
  GS_TRY(launch_dependent(k_lookup_keys, blocks_for(n), kThreads, 0, s, ids, n_ids, index, n, rows,
                          w.keys, w.order, dev_status));
  GS_LAUNCH_CHECK();
  return gs_sort_keys32(nullptr, w.keys, w.order, n, 0, key_bits(rows), 0, w.sort, w.sort_bytes,
                        dev_status, s);
}

template <class T, int V>
gs_status run_sums(const T* g, int64_t rs, int64_t n, int cols, float scale, float* dt, int64_t ld,
                   bool accumulate, const LookupWs& w, cudaStream_t s) {
  const int nv = (cols + V - 1) / V;
  int R = chunk_of(n, nv);
  int64_t m = n, chunks = (m + R - 1) / R;
  if (chunks * nv > (int64_t)INT32_MAX * kThreads) return GS_ERR_UNSUPPORTED;
  GS_TRY(launch_dependent(k_run_sums<T, V>, blocks_for(chunks * nv), kThreads, 0, s, w.keys, w.order,
                          m, R, g, rs, cols, Div((uint32_t)nv), scale, dt, ld, accumulate, w.pkey[0],
                          w.psum[0], w.ldp));
  GS_LAUNCH_CHECK();
  const int nv4 = (cols + 3) / 4;
  for (int from = 0; chunks > 1; from ^= 1) {
    m = 2 * chunks;
    chunks = (m + kPartChunk - 1) / kPartChunk;
    GS_TRY(launch_dependent(k_run_sums<float, 4>, blocks_for(chunks * nv4), kThreads, 0, s,
                            w.pkey[from], nullptr, m, kPartChunk, w.psum[from], w.ldp, cols,
                            Div((uint32_t)nv4), scale, dt, ld, accumulate, w.pkey[from ^ 1],
                            w.psum[from ^ 1], w.ldp));
    GS_LAUNCH_CHECK();
  }
  return GS_OK;
}

// Elements of size es that may move together: a divisor of cols and the
// stride that keeps every vector of the matrix aligned, at most `most`.
int vector_of(const void* p, int64_t ld, int cols, int es, int most) {
  int v = most;
  while (v > 1 && (cols % v || ld % v || !aligned(p, (size_t)v * es))) v >>= 1;
  return v;
}

template <class TT, class TO, int V>
gs_status launch_rows(const gs_matrix* t, const int32_t* ids, int64_t n_ids, const int32_t* index,
                      float scale, const gs_matrix* o, int32_t* dev_status, cudaStream_t s) {
  const int nv = o->cols / V;
  int items = kThreads * kRowIlp / nv;
  if (items < 1) items = 1;
  const int64_t blocks = (o->rows + items - 1) / items;
  k_lookup_rows<TT, TO, V><<<(unsigned)blocks, kThreads, 0, s>>>(
      static_cast<const TT*>(t->data), t->row_stride, t->rows, ids, n_ids, index, scale,
      static_cast<TO*>(o->data), o->rows, o->row_stride, Div((uint32_t)nv), items, dev_status);
  GS_LAUNCH_CHECK();
  return GS_OK;
}

template <class TT, class TO>
gs_status lookup_by(const gs_matrix* t, const int32_t* ids, int64_t n_ids, const int32_t* index,
                    float scale, const gs_matrix* o, int32_t* dev_status, cudaStream_t s) {
  if (o->col_stride != 1) {
    constexpr int V = 16 / sizeof(TT);
    const int cols = o->cols, words = (cols * (int)sizeof(TT) + 3) / 4;
    const int al = vector_of(t->data, t->row_stride, cols, sizeof(TT), 2 * V);
    const unsigned blocks = blocks_for(o->rows);
    if (al >= V && words > 8) {
      const unsigned groups = (unsigned)((o->rows + 32 * kStageWarps - 1) / (32 * kStageWarps));
      k_lookup_planes_staged<TT, TO><<<groups, 32 * kStageWarps, 0, s>>>(
              static_cast<const TT*>(t->data), t->row_stride, t->rows, cols, ids, n_ids, index,
              scale, static_cast<TO*>(o->data), o->rows, o->col_stride, dev_status);
      GS_LAUNCH_CHECK();
      return GS_OK;
    }
#define GS_LOOKUP_PLANES(NW, AL)                                                              \
  k_lookup_planes<TT, TO, NW, AL><<<blocks, kThreads, 0, s>>>(                                \
      static_cast<const TT*>(t->data), t->row_stride, t->rows, cols, ids, n_ids, index, scale, \
      static_cast<TO*>(o->data), o->rows, o->col_stride, dev_status)
    if (words <= 16) {
      if (al == 2 * V) GS_LOOKUP_PLANES(16, 32);
      else if (al == V) GS_LOOKUP_PLANES(16, 16);
      else GS_LOOKUP_PLANES(16, 0);
    } else {
      if (al == 2 * V) GS_LOOKUP_PLANES(48, 32);
      else if (al == V) GS_LOOKUP_PLANES(48, 16);
      else GS_LOOKUP_PLANES(48, 0);
    }
#undef GS_LOOKUP_PLANES
    GS_LAUNCH_CHECK();
    return GS_OK;
  }
  // both sides move v elements at a time, in at most 16 bytes
  constexpr int most = 16 / (sizeof(TT) > sizeof(TO) ? sizeof(TT) : sizeof(TO));
  const int vt = vector_of(t->data, t->row_stride, t->cols, sizeof(TT), most);
  const int vo = vector_of(o->data, o->row_stride, o->cols, sizeof(TO), most);
  const int v = vt < vo ? vt : vo;
  if constexpr (most == 8)
    if (v == 8) return launch_rows<TT, TO, 8>(t, ids, n_ids, index, scale, o, dev_status, s);
  if (v == 4) return launch_rows<TT, TO, 4>(t, ids, n_ids, index, scale, o, dev_status, s);
  if (v == 2) return launch_rows<TT, TO, 2>(t, ids, n_ids, index, scale, o, dev_status, s);
  return launch_rows<TT, TO, 1>(t, ids, n_ids, index, scale, o, dev_status, s);
}

template <class TT>
gs_status lookup_to(const gs_matrix* t, const int32_t* ids, int64_t n_ids, const int32_t* index,
                    float scale, const gs_matrix* o, int32_t* dev_status, cudaStream_t s) {
  switch (o->dtype) {
    case GS_F32: return lookup_by<TT, float>(t, ids, n_ids, index, scale, o, dev_status, s);
    case GS_F16: return lookup_by<TT, __half>(t, ids, n_ids, index, scale, o, dev_status, s);
    default: return lookup_by<TT, __nv_bfloat16>(t, ids, n_ids, index, scale, o, dev_status, s);
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
  if (n < 0 || n > (int64_t)INT32_MAX || rows < 1 || rows > (int64_t)INT32_MAX || cols < 1) return 0;
  const size_t b = carve_lookup(nullptr, 0, n, rows, cols, planes ? 4 : 0).bytes;
  return b ? b : 256;
}

extern "C" gs_status gs_lookup_plan(const int32_t* ids, int64_t n_ids, const int32_t* index,
                                    int64_t n, int64_t rows, int32_t cols, void* ws, size_t ws_bytes,
                                    int32_t* dev_status, gs_stream stream) {
  const gs_status st = check_ids(ids, n_ids, index, n);
  if (st != GS_OK) return st;
  if (rows < 1 || rows > (int64_t)INT32_MAX || cols < 1) return GS_ERR_ARG;
  if (n == 0) return GS_OK;
  const LookupWs w = carve_lookup(ws, ws_bytes, n, rows, cols, 0);
  if (!ws || w.bytes > ws_bytes || ws_bytes < 256) return GS_ERR_CAPACITY;
  if (!aligned(ws, 256)) return GS_ERR_ARG;
  if (n <= kSmallItems) return GS_OK;  // such gradients need no order
  return plan_lookup(ids, n_ids, index, n, rows, w, dev_status, to_stream(stream));
}

namespace gs {
namespace {

template <class T, int V>
gs_status small_grad(const gs_matrix* g, const int32_t* ids, int64_t n_ids, const int32_t* index,
                     float scale, const gs_matrix* dtable, bool accumulate, int32_t* dev_status,
                     cudaStream_t s) {
  // as many blocks as the table has 4096-element pieces, at most four per SM
  const int64_t rows = dtable->rows;
  int64_t blocks = (rows * dtable->cols + 4095) / 4096;
  if (blocks > 148 * 4) blocks = 148 * 4;
  if (blocks > rows) blocks = rows;
  const int64_t per = (rows + blocks - 1) / blocks;
  blocks = (rows + per - 1) / per;
  GS_TRY(launch_dependent(k_small_grad<T, V>, (unsigned)blocks, kThreads, 0, s,
                          static_cast<const T*>(g->data), g->row_stride, g->col_stride, g->cols, ids,
                          n_ids, index, (int)g->rows, scale, static_cast<float*>(dtable->data),
                          dtable->row_stride, rows, per, accumulate, dev_status));
  GS_LAUNCH_CHECK();
  return GS_OK;
}

template <class T>
gs_status lookup_grad(const gs_matrix* g, const int32_t* ids, int64_t n_ids, const int32_t* index,
                      float scale, const gs_matrix* dtable, bool accumulate, const LookupWs& w,
                      int32_t* dev_status, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int64_t n = g->rows;
  const int cols = g->cols;
  const T* data = static_cast<const T*>(g->data);
  const bool planes = g->col_stride != 1;
  const bool vec = !planes && vector_of(data, g->row_stride, cols, sizeof(T), V) == V;
  if (n <= kSmallItems)
    return vec ? small_grad<T, V>(g, ids, n_ids, index, scale, dtable, accumulate, dev_status, s)
               : small_grad<T, 1>(g, ids, n_ids, index, scale, dtable, accumulate, dev_status, s);
  float* dt = static_cast<float*>(dtable->data);
  const int64_t ld = dtable->row_stride;
  if (planes) {
    const int vecs = (cols + V - 1) / V;
    GS_TRY(launch_dependent(k_planes_to_rows<T>,
                            (unsigned)((n + 32 * kStageWarps - 1) / (32 * kStageWarps)),
                            32 * kStageWarps, 0, s, data, g->col_stride, cols, n, w.rows, vecs));
    GS_LAUNCH_CHECK();
    return run_sums<T, V>(reinterpret_cast<const T*>(w.rows), (int64_t)vecs * V, n, cols, scale, dt,
                          ld, accumulate, w, s);
  }
  return vec ? run_sums<T, V>(data, g->row_stride, n, cols, scale, dt, ld, accumulate, w, s)
             : run_sums<T, 1>(data, g->row_stride, n, cols, scale, dt, ld, accumulate, w, s);
}

}  // namespace
}  // namespace gs

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
  const int planes_es = g->col_stride != 1 ? (int)type_size(g->dtype) : 0;
  const LookupWs w = carve_lookup(ws, ws_bytes, n, rows, g->cols, planes_es);
  if (n > 0) {
    if (!ws || w.bytes > ws_bytes || ws_bytes < 256) return GS_ERR_CAPACITY;
    if (!aligned(ws, 256)) return GS_ERR_ARG;
  }
  const bool accumulate = (flags & GS_LOOKUP_ACCUMULATE) != 0;
  if (!accumulate && (n == 0 || n > kSmallItems))
    GS_TRY(cudaMemset2DAsync(dtable->data, dtable->row_stride * 4, 0, (size_t)g->cols * 4, rows, s));
  if (n == 0) return GS_OK;
  if (!(flags & GS_LOOKUP_PLANNED) && n > kSmallItems) {
    const gs_status ps = plan_lookup(ids, n_ids, index, n, rows, w, dev_status, s);
    if (ps != GS_OK) return ps;
  }
  const float sc = (float)scale;
  switch (g->dtype) {
    case GS_F32: return lookup_grad<float>(g, ids, n_ids, index, sc, dtable, accumulate, w, dev_status, s);
    case GS_F16: return lookup_grad<__half>(g, ids, n_ids, index, sc, dtable, accumulate, w, dev_status, s);
    default: return lookup_grad<__nv_bfloat16>(g, ids, n_ids, index, sc, dtable, accumulate, w, dev_status, s);
  }
}
