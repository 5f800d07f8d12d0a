// Embedding lookup with a scale, and its gradient by sorted ids.
//
// A table of K rows shared by n items (a colour codebook shared by the
// Gaussians, a per-view embedding): out[j] = scale * table[id_j], and
//   dtable[k] = scale * sum over {j : id_j = k} of g[j].
// gs_grad_accumulate scatters gradients whose indices are all different;
// here an index may occur any number of times.  The gradient has three forms,
// chosen by sizes and layout, none with float atomics, so that equal inputs
// give equal bits: few items in one launch (k_small_grad), tables that fit in
// shared memory (k_private_sums), and items sorted by id whose runs are then
// summed (k_sort_*, k_planes_to_rows, k_run_sums).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

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
// flight.  A block takes kThreads * kRowIlp consecutive vectors.  Bound by HBM
// and by the latency of id and row: 2M x 64 fp32 take 88 us (6.1 TB/s), 2M x
// 27, whose rows are not aligned to vectors, 102 us (2.3 TB/s; 16 bytes of out
// per thread, element by element: 111); a call of 33 x 32 is 3.2 us on the
// device.  16-byte stores of fp32 are marked as streaming (118 us without),
// the others not: it costs 16-bit outputs 8 to 15%.
constexpr int kRowIlp = 4;
template <class TT, class TO, int V>
__global__ void __launch_bounds__(kThreads)
k_lookup_rows(const TT* __restrict__ table, int64_t ld, int64_t rows,
              const int32_t* __restrict__ ids, int64_t n_ids, const int32_t* __restrict__ index,
              float scale, TO* __restrict__ out, int64_t n, int64_t rs, Div nv, int items,
              int32_t* dev_status) {
  wait_for_prior_grids();
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
      Pack<TO, V>* to = reinterpret_cast<Pack<TO, V>*>(out + (j0 + at[k]) * rs + c[k]);
      if constexpr (sizeof(w) == 16 && sizeof(TO) == 4)
        __stcs(reinterpret_cast<uint4*>(to), *reinterpret_cast<const uint4*>(&w));
      else
        *to = w;
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
// element.  1M x 27 from a bf16 table take 22 us (5.1 TB/s); 26 without the
// stores marked as streaming, 60 with one load per element and a turn in
// shared memory.
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
  wait_for_prior_grids();
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= n) return;
  const int32_t id = id_of(ids, n_ids, index, j, rows, dev_status);
  const bool has = id >= 0;
  TO* o = out + j;
  uint32_t w[NL];
  const auto store = [&](int c) {
    __stcs(o, from_f<TO>(has ? scale * element<TT>(w, c) : 0.f));
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

// out in planes, rows of more than 64 bytes on 16-byte boundaries: a block
// fetches the rows of kTurnItems items (192 bytes of them at a time) into
// shared memory by one bulk copy each, and a warp writes four (eight) planes'
// pieces of 128 items from there, 16 bytes of a row at a time.  The row pitch
// of 4 words more than a multiple of 16 keeps those reads free of bank
// conflicts.  6M x 48 fp32 take 218 us (5.5 TB/s); 271 with 16-byte
// asynchronous copies, 309 with a lane reading its own row as above, 310 with
// the planes' pieces turned once more and stored in bulk.  A lane's own row
// costs a request for every 32 bytes; up to 64 bytes that is the faster form
// (1M x 16: 19 us against 28 by this one, 1M x 12: 18 against 28).  No unit is
// saturated (1.5M x 48: the SMs' requests to L2 busy 62% of the cycles, DRAM
// 48%, issue 51%): a block's ids, its rows and its stores wait for one
// another, and shared memory holds four blocks to an SM.
constexpr int kTurnItems = 256;
constexpr int kStageVecs = 12, kStagePitch = 4 * kStageVecs + 4;  // words
constexpr size_t kStageSmem = sizeof(uint32_t) * kTurnItems * kStagePitch;

__device__ __forceinline__ void copy_16_async(void* smem, const void* p, bool has) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(smem)), "l"(p),
               "r"(has ? 16 : 0)
               : "memory");
}

// Waits (bounded) for the bulk copies of the barrier's phase; on expiry sets
// the flag, waits once more so that none lands in memory given up, and
// returns false.
__device__ __forceinline__ bool copies_landed(unsigned long long* bar, unsigned phase,
                                              int32_t* dev_status) {
  if (mbar_wait(bar, phase)) return true;
  dev_flag(dev_status, GS_DEV_TIMEOUT);
  mbar_wait(bar, phase);
  return false;
}

template <class TT, class TO>
__global__ void __launch_bounds__(kThreads)
k_lookup_planes_staged(const TT* __restrict__ table, int64_t ld, int64_t rows, int cols,
                       const int32_t* __restrict__ ids, int64_t n_ids,
                       const int32_t* __restrict__ index, float scale, TO* __restrict__ out,
                       int64_t n, int64_t cs, int32_t* dev_status) {
  constexpr int V = 16 / sizeof(TT), W = kThreads / 32, PIECE = 128;
  static_assert(kThreads == kTurnItems, "a thread for each item's id");
  extern __shared__ __align__(16) uint32_t s_rows[];
  __shared__ int16_t s_from[kTurnItems];  // the row that holds an item's values; -1: zeros
  __shared__ unsigned long long s_bar;
  unsigned phase = 0;
  if (threadIdx.x == 0) {
    mbar_init(&s_bar, 1);
    fence_mbar_init();
  }
  wait_for_prior_grids();
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int64_t j0 = (int64_t)blockIdx.x * kTurnItems;
  const int items = (int)min((int64_t)kTurnItems, n - j0);
  const int32_t id = t < items ? id_of(ids, n_ids, index, j0 + t, rows, dev_status) : -1;
  // lanes with the same id share the first one's copy: a row that many items
  // use would otherwise be fetched from one place of L2 by all SMs at once
  // (1M items of a one-row table of 64 columns: 45 us, 584 without this)
  const int leader = __ffs(__match_any_sync(0xffffffffu, id)) - 1;
  const bool fetch = id >= 0 && leader == lane;
  s_from[t] = id >= 0 ? (int16_t)(t - lane + leader) : -1;
  __syncthreads();
  for (int c0 = 0; c0 < cols; c0 += kStageVecs * V) {
    const int nv = min(kStageVecs, (cols - c0) / V);
    // a row per thread: one bulk copy
    const int copies = __syncthreads_count(fetch);
    if (t == 0) mbar_arrive_expect_tx(&s_bar, (unsigned)(copies * nv * 16));
    __syncthreads();
    if (fetch) bulk_load(s_rows + t * kStagePitch, table + (int64_t)id * ld + c0, nv * 16, &s_bar);
    if (!copies_landed(&s_bar, phase, dev_status)) return;
    phase ^= 1;
    __syncthreads();
    for (int u = w; u < nv * (kTurnItems / PIECE); u += W) {
      const int q = u / (kTurnItems / PIECE);
      TO* o = out + (int64_t)(c0 + q * V) * cs + j0;
#pragma unroll
      for (int k = 0; k < PIECE / 32; ++k) {
        const int j = u % (kTurnItems / PIECE) * PIECE + k * 32 + lane;
        if (j >= items) break;
        const int from = s_from[j];
        const bool has = from >= 0;
        uint32_t x[4];
        *reinterpret_cast<uint4*>(x) =
            *reinterpret_cast<const uint4*>(s_rows + (has ? from : j) * kStagePitch + 4 * q);
#pragma unroll
        for (int i = 0; i < V; ++i)
          __stcs(o + i * cs + j, from_f<TO>(has ? scale * element<TT>(x, i) : 0.f));
      }
    }
    __syncthreads();
  }
}

// Stable radix sort of the gradient's items by id: pairs (id, item), digits
// of up to 10 bits, most often one or two passes.  A pass counts the digits
// of each tile of kSortTile items, scans the counts along the tiles, and
// scatters.  The first pass reads the ids themselves.  An item without a row
// takes the last id and item -1, which adds nothing, so that the keys need no
// bit more than the rows do.  Bound by the latency of the ranking in shared
// memory: 2.5M items over 2^16 rows take 59 us in the six kernels; the
// library's general 32-bit sort took 127 (8 bits per pass, an even number of
// passes, a histogram before them, tiles of 4096).  Ranks by ballots over the
// digit's bits: 20 us a pass, 29 with the match instruction.
// For few items the kernels' launches are what costs: up to kFewTiles tiles
// the scatter sums the tiles' counts itself and counts the next pass's digits
// as it writes (integer atomics: the counts do not depend on their order), so
// that a pass is one launch after the first.  100K items x 16 take 33 us so,
// 40 without; 300K take 45 and 42.
constexpr int kFewTiles = 64;
constexpr int kSortItems = 8, kSortTile = kThreads * kSortItems, kMaxDigit = 10;

struct Ids {
  const int32_t* ids;
  const int32_t* index;
  int64_t n_ids, rows;
};

// counts[digit][tile] (few tiles: counts[tile][digit]); the first pass also
// writes the pairs and clears the `later` passes' counts, which follow, and
// `zeros` floats of dtable
template <bool FIRST>
__global__ void __launch_bounds__(kThreads)
k_sort_count(const __grid_constant__ Ids src, uint2* __restrict__ pairs, int64_t n, int shift,
             int bits, uint32_t* __restrict__ counts, bool few, int later, float* __restrict__ dtable,
             int64_t zeros, int32_t* dev_status) {
  __shared__ uint32_t s_hist[1 << kMaxDigit];
  wait_for_prior_grids();
  const int t = threadIdx.x, bins = 1 << bits;
  for (int d = t; d < bins; d += kThreads) s_hist[d] = 0;
  __syncthreads();
  const int64_t j0 = (int64_t)blockIdx.x * kSortTile + t;
  uint32_t key[kSortItems];
  if (FIRST) {
    // all positions, then all ids in flight
    int64_t at[kSortItems];
    int32_t id[kSortItems];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const int64_t j = j0 + i * kThreads;
      at[i] = j < n ? (src.index ? (int64_t)src.index[j] : j) : -1;
    }
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const bool in = at[i] >= 0 && (!src.index || at[i] < src.n_ids);
      bad |= j0 + i * kThreads < n && !in;
      id[i] = in ? src.ids[at[i]] : -1;
    }
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const int64_t j = j0 + i * kThreads;
      if (id[i] >= src.rows) {
        bad = true;
        id[i] = -1;
      }
      key[i] = id[i] >= 0 ? (uint32_t)id[i] : (uint32_t)(src.rows - 1);
      if (j < n) pairs[j] = make_uint2(key[i], id[i] >= 0 ? (uint32_t)j : 0xffffffffu);
    }
    if (bad) dev_flag(dev_status, GS_DEV_BOUNDS);
    const int64_t quads = zeros / 4, at0 = (int64_t)blockIdx.x * kThreads + t;
    for (int64_t i = at0; i < quads; i += (int64_t)gridDim.x * kThreads)
      reinterpret_cast<uint4*>(dtable)[i] = make_uint4(0, 0, 0, 0);
    if (at0 < zeros % 4) dtable[4 * quads + at0] = 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const int64_t j = j0 + i * kThreads;
      if (j < n) key[i] = pairs[j].x;
    }
  }
#pragma unroll
  for (int i = 0; i < kSortItems; ++i)
    if (j0 + i * kThreads < n) atomicAdd(&s_hist[(key[i] >> shift) & (bins - 1)], 1u);
  __syncthreads();
  for (int d = t; d < bins; d += kThreads)
    counts[few ? (int64_t)blockIdx.x * bins + d : (int64_t)d * gridDim.x + blockIdx.x] = s_hist[d];
  if (FIRST && later > 0) {
    const int64_t size = (int64_t)gridDim.x * bins;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + t; i < size * later; i += (int64_t)gridDim.x * kThreads)
      counts[size + i] = 0;
  }
}

// counts of digit blockIdx.x -> exclusive sums over the tiles; total[digit]
__global__ void __launch_bounds__(kThreads)
k_sort_scan(uint32_t* __restrict__ counts, int64_t tiles, uint32_t* __restrict__ total) {
  __shared__ uint32_t s_scan[kThreads / 32 + 1];
  wait_for_prior_grids();
  uint32_t* c = counts + (int64_t)blockIdx.x * tiles;
  uint32_t base = 0;
  for (int64_t i0 = 0; i0 < tiles; i0 += kThreads * 4) {
    const int64_t i = i0 + threadIdx.x * 4;
    uint32_t v[4], sum = 0, all;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = i + k < tiles ? c[i + k] : 0;
      sum += v[k];
    }
    uint32_t at = base + block_exclusive_scan<uint32_t, kThreads / 32>(sum, s_scan, &all);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < tiles) {
        c[i + k] = at;
        at += v[k];
      }
    base += all;
  }
  if (threadIdx.x == 0) total[blockIdx.x] = base;
}

size_t scatter_smem(int bits) {
  return sizeof(uint2) * kSortTile + ((size_t)1 << bits) * (2 * sizeof(uint32_t) + 2 * (kThreads / 32));
}

// FEW: counts[tile][digit] of this pass; next: those of the next pass (or null)
template <bool FEW>
__global__ void __launch_bounds__(kThreads, 3)
k_sort_scatter(const uint2* __restrict__ pairs, int64_t n, int shift, int bits,
               const uint32_t* __restrict__ counts, const uint32_t* __restrict__ total,
               uint32_t* __restrict__ next, uint2* __restrict__ out) {
  constexpr int kWarps = kThreads / 32, kPer = (1 << kMaxDigit) / kThreads;
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ unsigned long long s_scan[kWarps + 1];
  const int bins = 1 << bits;
  uint2* s_pair = reinterpret_cast<uint2*>(s_raw);
  uint32_t* s_loc = reinterpret_cast<uint32_t*>(s_pair + kSortTile);  // digit's start in the tile
  uint32_t* s_base = s_loc + bins;                                    // ... in the output, less that
  uint16_t* s_hist = reinterpret_cast<uint16_t*>(s_base + bins);      // [warp][digit]
  wait_for_prior_grids();
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int64_t j0 = (int64_t)blockIdx.x * kSortTile;
  const int items = (int)min((int64_t)kSortTile, n - j0);
  uint2 p[kSortItems];
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {  // a warp's items are neighbours
    const int e = w * 32 * kSortItems + i * 32 + lane;
    if (e < items) p[i] = pairs[j0 + e];
    else p[i] = make_uint2(0xffffffffu, 0);  // behind the last item: behind all of the last digit
  }
  // thread t has `per` neighbouring digits
  const int per = (bins + kThreads - 1) / kThreads;
  uint32_t tot[kPer], cnt[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int d = t * per + i;
    const bool in = i < per && d < bins;
    if (!FEW) {
      tot[i] = in ? total[d] : 0;
      cnt[i] = in ? counts[(int64_t)d * gridDim.x + blockIdx.x] : 0;
    } else {
      tot[i] = cnt[i] = 0;
      if (in) {
        for (int k0 = 0; k0 < (int)gridDim.x; k0 += 16) {
          uint32_t c[16];  // all in flight, the last ones too
#pragma unroll
          for (int k = 0; k < 16; ++k) c[k] = k0 + k < (int)gridDim.x ? counts[(k0 + k) * bins + d] : 0;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            tot[i] += c[k];
            if (k0 + k < (int)blockIdx.x) cnt[i] += c[k];
          }
        }
      }
    }
  }
  for (int i = t; i < bins * kWarps / 2; i += kThreads) reinterpret_cast<uint32_t*>(s_hist)[i] = 0;
  __syncthreads();
  // rank of an item among its warp's items with the same digit
  uint16_t rank[kSortItems];
  uint16_t* hist = s_hist + w * bins;
  unsigned same_of[kSortItems];
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) same_of[i] = 0xffffffffu;
  for (int k = shift; k < shift + bits; ++k)
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const bool one = (p[i].x >> k) & 1;
      const unsigned bal = __ballot_sync(0xffffffffu, one);
      same_of[i] &= one ? bal : ~bal;
    }
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const uint32_t d = (p[i].x >> shift) & (bins - 1);
    const unsigned same = same_of[i];
    const int before = __popc(same & ((1u << lane) - 1)), had = hist[d];
    rank[i] = (uint16_t)(had + before);
    __syncwarp();
    if (before == 0) hist[d] = (uint16_t)(had + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  uint32_t local = 0, global = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int d = t * per + i;
    if (i < per && d < bins) {
      uint32_t run = 0;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const uint32_t c = s_hist[k * bins + d];
        s_hist[k * bins + d] = (uint16_t)run;
        run += c;
      }
      s_loc[d] = local;
      s_base[d] = global + cnt[i];
      local += run;
      global += tot[i];
    }
  }
  // both scans at once: a tile has at most 2^11 items, the list less than 2^31
  unsigned long long all;
  const unsigned long long both = block_exclusive_scan<unsigned long long, kWarps>(
      (unsigned long long)local << 32 | global, s_scan, &all);
  for (int d = t * per; d < min(bins, (t + 1) * per); ++d) {
    s_loc[d] += (uint32_t)(both >> 32);
    s_base[d] += (uint32_t)both - s_loc[d];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const uint32_t d = (p[i].x >> shift) & (bins - 1);
    s_pair[s_loc[d] + hist[d] + rank[i]] = p[i];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = t + k * kThreads;
    if (i < items) {
      const uint2 x = s_pair[i];
      const uint32_t at = s_base[(x.x >> shift) & (bins - 1)] + i;
      out[at] = x;
      if (FEW && next)
        atomicAdd(&next[at / kSortTile * bins + ((x.x >> (shift + bits)) & (bins - 1))], 1u);
    }
  }
}

// Planes to rows (pitch `vecs` 16-byte vectors, columns past the last one
// zero): the sums below read whole rows in the order of their ids, and a row
// in planes costs a 32-byte sector for every element.  A block copies
// kTurnItems items of up to 192 bytes' columns into shared memory, a plane's
// piece at a time, all in flight, and writes the rows as one contiguous piece.
// Bound by HBM: 2.5M x 48 fp32 take 170 us (5.6 TB/s read and written).  The
// pieces' length counts: 1 KB here, 181 us with 512 bytes, 207 with 128.
// 16-bit planes move two elements at a time: 1.5M x 48 fp16 take 60 us (4.9
// TB/s), 81 by single elements.
template <class T>
struct Turn {
  static constexpr int V = 16 / sizeof(T), kVecs = 12, kCols = kVecs * V;
  static constexpr int kPitch = kTurnItems + 4 / sizeof(T);  // odd in words
  static constexpr size_t kSmem = sizeof(T) * kCols * kPitch;
  static size_t smem(int vecs) { return vecs < kVecs ? sizeof(T) * vecs * V * kPitch : kSmem; }
};

template <class T>
__global__ void __launch_bounds__(kThreads)
k_planes_to_rows(const T* __restrict__ g, int64_t cs, int cols, int64_t n, uint4* __restrict__ out,
                 int vecs) {
  constexpr int V = Turn<T>::V, kVecs = Turn<T>::kVecs, P = Turn<T>::kPitch, W = kThreads / 32;
  extern __shared__ __align__(16) unsigned char s_raw[];
  T* s = reinterpret_cast<T*>(s_raw);
  wait_for_prior_grids();
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int64_t j0 = (int64_t)blockIdx.x * kTurnItems;
  const int items = (int)min((int64_t)kTurnItems, n - j0);
  // whether a 16-bit plane's piece starts half a word in: it lies the same way
  // in shared memory
  const unsigned start = (unsigned)((reinterpret_cast<uintptr_t>(g) >> 1) + j0), by = (unsigned)cs;
  const auto odd = [&](int c) { return sizeof(T) == 2 ? (int)((start + (unsigned)c * by) & 1u) : 0; };
  for (int v0 = 0; v0 < vecs; v0 += kVecs) {
    const int nv = min(kVecs, vecs - v0), c0 = v0 * V;
    for (int c = w; c < nv * V; c += W) {
      const T* p = g + (int64_t)(c0 + c) * cs + j0;
      T* d = s + c * P;
      if (c0 + c >= cols) {
        for (int j = lane; j < items; j += 32) d[odd(c0 + c) + j] = from_f<T>(0.f);
      } else if (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < kTurnItems / 32; ++k)
          if (lane + 32 * k < items)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(d + lane + 32 * k)),
                         "l"(p + lane + 32 * k)
                         : "memory");
      } else {  // two elements at a time, single ones at the plane piece's ends
        const int off = odd(c0 + c);
#pragma unroll
        for (int k = 0; k < kTurnItems / 64 + 1; ++k) {
          const int e = 2 * (lane + 32 * k) - off;
          if (e >= 0 && e + 1 < items) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(d + off + e)),
                         "l"(p + e)
                         : "memory");
          } else {
            if (e >= 0 && e < items) d[off + e] = p[e];
            if (e + 1 >= 0 && e + 1 < items) d[off + e + 1] = p[e + 1];
          }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    int r = t / nv, v = t - r * nv;
    const int dr = kThreads / nv, dv = kThreads - dr * nv;
    for (int e = t; e < items * nv; e += kThreads) {
      Pack<T, V> x;
#pragma unroll
      for (int i = 0; i < V; ++i) x.x[i] = s[(v * V + i) * P + odd(c0 + v * V + i) + r];
      *reinterpret_cast<Pack<T, V>*>(out + (j0 + r) * vecs + v0 + v) = x;
      r += dr;
      v += dv;
      if (v >= nv) {
        v -= nv;
        ++r;
      }
    }
    __syncthreads();
  }
}

// Sums of runs of equal keys over a list of n entries: the sorted items
// (FIRST: pairs of a key and a row of g) or partials (keys, entry r being row
// r).  A block takes E entries and copies their rows (`width` vectors of V
// columns) into shared memory, all in flight at once without a register held;
// then teams of `width` threads sum `len` entries each from there.  A run
// inside a team's entries goes to dtable.  What a team holds of a run that
// crosses its borders goes to a slot: slot 0 if the run came in from before,
// else slot 1; the team in which a run starts then adds the following teams'
// slots 0 in order.  Runs that cross the block's borders leave as partials:
// entry 2 block for a run that came in, 2 block + 1 for one that starts here
// and goes on; a block inside one run writes its sum at 2 block and zeros at
// 2 block + 1, so that a run's partials are neighbours.  Unused partials have
// the key kNoRow.  The same kernel sums the partials until one block is left.
// Bound by HBM at random rows: 2.5M x 48 fp32 take 123 us (3.9 TB/s; a row of
// 192 bytes costs 256 of DRAM traffic), 130 with the rows in registers, eight
// in flight; bands of columns small enough to stay in L2 between turning and
// summing were slower in all (576 us for 24 columns at a time against 498).
// d[0 .. V) (+)= scale * sum of the columns that exist; vec: 16-byte stores
template <int V>
__device__ __forceinline__ void to_row(float* d, const float* sum, int left, float scale,
                                       bool accumulate, bool vec) {
  if (V >= 4 && vec) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      if (i >= left) break;
      float4* p = reinterpret_cast<float4*>(d + i);
      float4 x = accumulate ? *p : make_float4(0.f, 0.f, 0.f, 0.f);
      if (accumulate) {
        x.x += scale * sum[i], x.y += scale * sum[i + 1];
        x.z += scale * sum[i + 2], x.w += scale * sum[i + 3];
      } else {
        x = make_float4(scale * sum[i], scale * sum[i + 1], scale * sum[i + 2], scale * sum[i + 3]);
      }
      *p = x;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < left) d[i] = accumulate ? d[i] + scale * sum[i] : scale * sum[i];
}

// V floats between registers and 16-byte aligned memory (any for V = 1)
template <int V>
__device__ __forceinline__ void put_floats(float* d, const float* v) {
  if (V == 1) *d = *v;
#pragma unroll
  for (int i = 0; i + 3 < V; i += 4)
    *reinterpret_cast<float4*>(d + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int V>
__device__ __forceinline__ void add_floats(float* v, const float* d) {
  if (V == 1) *v += *d;
#pragma unroll
  for (int i = 0; i + 3 < V; i += 4) {
    const float4 x = *reinterpret_cast<const float4*>(d + i);
    v[i] += x.x, v[i + 1] += x.y, v[i + 2] += x.z, v[i + 3] += x.w;
  }
}

constexpr int kMaxTeams = 128, kRunRowBytes = 40 * 1024, kRunEntries = 1024;

struct RunShape {
  int width, pitch, teams, entries, len, col_tiles, smem;  // pitch in bytes
  int64_t blocks;
  RunShape(int64_t n, int cols, int V, int es, bool first) {
    const int nv = (cols + V - 1) / V, most = V == 1 ? 64 : 16;
    col_tiles = (nv + most - 1) / most;
    width = (nv + col_tiles - 1) / col_tiles;
    pitch = V == 1 ? (width * es + 3) / 4 * 4 : 16 * (width | 1);
    teams = kThreads / width < kMaxTeams ? kThreads / width : kMaxTeams;
    // what fits, for the items no more than leaves two blocks for each SM
    int64_t e = kRunRowBytes / pitch, fill = n / (148 * 2);
    if (e > kRunEntries) e = kRunEntries;
    if (first && e > fill) e = fill < 64 ? 64 : fill;
    entries = (int)e;
    len = (entries + teams - 1) / teams;
    blocks = (n + entries - 1) / entries;
    smem = (entries * pitch + 15) / 16 * 16 + 2 * kThreads * V * 4 + entries * 8;
  }
};

template <class T, int V, bool FIRST>
__global__ void __launch_bounds__(kThreads)
k_run_sums(const uint2* __restrict__ pairs, const uint32_t* __restrict__ keys, int64_t n,
           const __grid_constant__ RunShape sh, const T* __restrict__ g, int64_t rs, int cols,
           float scale, float* __restrict__ dtable, int64_t ld, uint32_t rows, bool vec, bool accumulate,
           uint32_t* __restrict__ pkey, float* __restrict__ psum, int ldp, int32_t* dev_status) {
  extern __shared__ __align__(16) unsigned char s_row[];  // [entries][pitch]
  __shared__ bool s_start[kMaxTeams], s_whole[kMaxTeams];
  const int pitch = sh.pitch, len = sh.len;
  float* s_part = reinterpret_cast<float*>(s_row + (sh.entries * pitch + 15) / 16 * 16);
  uint32_t* s_key = reinterpret_cast<uint32_t*>(s_part + 2 * kThreads * V);
  int32_t* s_item = reinterpret_cast<int32_t*>(s_key + sh.entries);
  wait_for_prior_grids();
  const int t = threadIdx.x;
  const int64_t blk = blockIdx.x / sh.col_tiles, A = blk * sh.entries;
  const int m = (int)min((int64_t)sh.entries, n - A);
  const int v0 = (int)(blockIdx.x % sh.col_tiles) * sh.width;
  const int width = min(sh.width, (cols + V - 1) / V - v0);
  for (int i = t; i < m; i += kThreads) {
    if (FIRST) {
      // a kept order that is none (memory that no plan wrote) stays in bounds
      const uint2 p = pairs[A + i];
      const bool good = p.x < rows && ((int32_t)p.y < 0 || p.y < n);
      if (!good) dev_flag(dev_status, GS_DEV_BOUNDS);
      s_key[i] = good ? p.x : kNoRow;
      s_item[i] = good ? (int32_t)p.y : -1;
    } else {
      s_key[i] = keys[A + i];
    }
  }
  const auto key_at = [&](int64_t r) {
    const uint32_t k = FIRST ? pairs[r].x : keys[r];
    return FIRST && k >= rows ? kNoRow : k;
  };
  const uint32_t before = A > 0 ? key_at(A - 1) : kNoRow, after = A + m < n ? key_at(A + m) : kNoRow;
  __syncthreads();
  {
    int r = t / width, v = t - r * width;
    const int dr = kThreads / width, dv = kThreads - dr * width;
    for (int e = t; e < m * width; e += kThreads) {
      const int64_t j = FIRST ? (int64_t)s_item[r] : A + r;
      const bool has = FIRST ? j >= 0 : s_key[r] != kNoRow;
      const T* from = g + (has ? j : 0) * rs + (v0 + v) * V;
      if (V > 1) {
        copy_16_async(s_row + r * pitch + 16 * v, from, has);
      } else if (sizeof(T) == 4) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                         smem_addr(s_row + r * pitch + 4 * v)),
                     "l"(from), "r"(has ? 4 : 0)
                     : "memory");
      } else {
        reinterpret_cast<T*>(s_row + r * pitch)[v] = has ? *from : from_f<T>(0.f);
      }
      r += dr;
      v += dv;
      if (v >= width) {
        v -= width;
        ++r;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  const int used = (m + len - 1) / len;  // teams with entries
  const int team = t / width, tv = t - team * width, c = (v0 + tv) * V;
  const bool on = team < used;  // m <= teams * len of the full width, and width is at most that
  uint32_t k = kNoRow;
  bool head = false, start = false, whole = false;
  float sum[V];
  const auto to_table = [&](uint32_t key) {
    to_row<V>(dtable + (int64_t)key * ld + c, sum, cols - c, scale, accumulate, vec);
  };
  const auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.f;
  };
  const auto done = [&](bool tail) {
    if (k == kNoRow) return;
    if (!head && !tail) return to_table(k);
    put_floats<V>(s_part + (head ? 0 : kThreads * V) + t * V, sum);
    start = !head;
    whole = head && tail;
  };
  if (on) {
    const int a = team * len, b = min(a + len, m);
    k = s_key[a];
    head = k == (a > 0 ? s_key[a - 1] : before) && k != kNoRow;
    clear();
    for (int r = a; r < b; ++r) {
      const uint32_t kr = s_key[r];
      const Pack<T, V> x = *reinterpret_cast<const Pack<T, V>*>(s_row + r * pitch + tv * V * sizeof(T));
      if (kr != k) {
        done(false);
        k = kr;
        head = false;
        clear();
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += to_f(x.x[i]);
    }
    start = whole = false;  // of the last run: the first may have left a slot 0
    done(k == (b < m ? s_key[b] : after));
    if (tv == 0) {
      s_start[team] = start;
      s_whole[team] = whole;
    }
  }
  __syncthreads();
  if (!on) return;
  // runs that came into the block (team 0), and that start in this team
  bool used0 = false;
  const auto leave = [&](int slot, uint32_t key, bool zero) {
    const int64_t p = 2 * blk + slot;
    if (c == 0) pkey[p] = key;
    const float none[V] = {};
    put_floats<V>(psum + p * ldp + c, zero ? none : sum);
  };
  const auto add_following = [&](int u) {  // -> true if the run leaves the block
    for (; u < used; ++u) {
      add_floats<V>(sum, s_part + (u * width + tv) * V);
      if (!s_whole[u]) return false;
    }
    return true;
  };
  const auto load = [&](int slot) {
    clear();
    add_floats<V>(sum, s_part + slot * kThreads * V + t * V);
  };
  if (team == 0 && before != kNoRow && before == s_key[0]) {
    load(0);
    const bool through = s_whole[0] && add_following(1);
    leave(0, before, false);
    if (through) leave(1, before, true);
    used0 = true;
  }
  if (s_start[team]) {
    load(1);
    if (add_following(team + 1)) leave(1, k, false);
    else to_table(k);
  }
  // the partials that nothing set: entry 0 is team 0's, entry 1 whoever's run
  // leaves the block
  if (c == 0) {
    if (team == 0 && !used0) pkey[2 * blk] = kNoRow;
    if (team == used - 1 && (after == kNoRow || after != s_key[m - 1])) pkey[2 * blk + 1] = kNoRow;
  }
}

// Up to kSmallItems items, in one launch: a block owns a range of up to
// kSmallRows of the table's rows and of the columns.  It picks the items with
// ids in its range (in order), sorts them by id in shared memory (the rank of
// an item among its warp's equal ids from ballots over the id's bits, as in
// the sort above), sums the runs of equal ids with teams of threads, each a
// stretch of the sorted list, joins the teams' partial runs in order, and
// clears the rows that nothing used.  Every block reads all ids.  Bound by
// latency: 37 x 16 for 100 rows take 5.3 us on the device.
constexpr int kSmallItems = 2048, kSmallPer = kSmallItems / kThreads;
constexpr int kSmallTeams = 64, kSmallRows = 1024;

template <class T, int V>
__global__ void __launch_bounds__(kThreads)
k_small_grad(const T* __restrict__ g, int64_t rs, int64_t cs, int cols, int share,
             unsigned col_tiles, const int32_t* __restrict__ ids, int64_t n_ids,
             const int32_t* __restrict__ index, int n, float scale, float* __restrict__ dtable,
             int64_t ld, int64_t rows, int per, bool accumulate, int32_t* dev_status) {
  constexpr int W = kThreads / 32;
  __shared__ int32_t s_key[kSmallItems];
  __shared__ uint16_t s_item[kSmallItems];
  __shared__ int s_scan[W + 1];
  __shared__ int32_t s_pk[2 * kSmallTeams];
  __shared__ uint32_t s_loc[kSmallRows];
  // the sort's counts [warp][row], then the teams' partial sums
  __shared__ __align__(16) unsigned char s_both[2 * kSmallRows * W];
  static_assert(sizeof(float) * 2 * kThreads * V <= sizeof(s_both), "partial sums fit");
  uint16_t* s_hist = reinterpret_cast<uint16_t*>(s_both);
  float* s_part = reinterpret_cast<float*>(s_both);
  wait_for_prior_grids();
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int64_t k0 = (int64_t)(blockIdx.x / col_tiles) * per, k1 = min(k0 + per, rows);
  // this block's vectors of V columns
  const int nv = (cols + V - 1) / V, first = (int)(blockIdx.x % col_tiles) * share;
  const int last = min(first + share, nv);
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
    const int c0 = first * V, width = min(last * V, cols) - c0;
    float* d = dtable + k0 * ld + c0;
    if (width == ld) {
      const int64_t total = (k1 - k0) * ld;
      for (int64_t i = t; i < total; i += kThreads) d[i] = 0.f;
    } else {
      // 32 columns of a warp's row at a time
      for (int64_t k = w; k < k1 - k0; k += W)
        for (int c = lane; c < width; c += 32) d[k * ld + c] = 0.f;
    }
  }
  int m;
  int at = block_exclusive_scan<int, W>(mine, s_scan, &m);
  if (m == 0) return;
#pragma unroll
  for (int i = 0; i < kSmallPer; ++i)
    if (key[i] >= 0) {
      s_key[at] = key[i];
      s_item[at++] = (uint16_t)(t * kSmallPer + i);
    }
  const int digits = (int)(k1 - k0);
  if (digits > 1)
    for (int i = t; i < (digits * W + 1) / 2; i += kThreads) reinterpret_cast<uint32_t*>(s_hist)[i] = 0;
  __syncthreads();  // also: the zeros above are ordered before the sums below
  if (digits > 1) {
    const int bits = 32 - __clz(digits - 1), rounds = (m + kThreads - 1) / kThreads;
    uint16_t* hist = s_hist + w * digits;
    int32_t mk[kSmallPer];
    uint16_t mi[kSmallPer], rank[kSmallPer];
#pragma unroll
    for (int i = 0; i < kSmallPer; ++i) {  // a warp's items are neighbours
      if (i >= rounds) break;
      const int e = (w * rounds + i) * 32 + lane;
      const bool in = e < m;
      mk[i] = in ? s_key[e] : 0;
      mi[i] = in ? s_item[e] : 0;
      unsigned same = __ballot_sync(0xffffffffu, in);
      for (int k = 0; k < bits; ++k) {
        const bool one = (mk[i] >> k) & 1;
        const unsigned bal = __ballot_sync(0xffffffffu, one);
        same &= one ? bal : ~bal;
      }
      const int before = __popc(same & ((1u << lane) - 1)), had = in ? hist[mk[i]] : 0;
      rank[i] = (uint16_t)(had + before);
      __syncwarp();
      if (in && before == 0) hist[mk[i]] = (uint16_t)(had + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    const int each = (digits + kThreads - 1) / kThreads;
    int local = 0, all;
    for (int d = t * each; d < min(digits, (t + 1) * each); ++d) {
      int run = 0;
      for (int k = 0; k < W; ++k) {
        const int c = s_hist[k * digits + d];
        s_hist[k * digits + d] = (uint16_t)run;
        run += c;
      }
      s_loc[d] = local;
      local += run;
    }
    const int base = block_exclusive_scan<int, W>(local, s_scan, &all);
    for (int d = t * each; d < min(digits, (t + 1) * each); ++d) s_loc[d] += base;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSmallPer; ++i)
      if (i < rounds && (w * rounds + i) * 32 + lane < m) {
        const int p = s_loc[mk[i]] + hist[mk[i]] + rank[i];
        s_key[p] = mk[i];
        s_item[p] = mi[i];
      }
    __syncthreads();
  }
  const int mine_v = last - first;
  int teams = mine_v < kThreads ? kThreads / mine_v : 1;
  teams = min(teams, min(kSmallTeams, (m + 3) / 4));
  const int len = (m + teams - 1) / teams;
  const int width = min(mine_v, kThreads);  // vectors of a row at a time
  const int team = t / width, tv = t - team * width;
  for (int v0 = first; v0 < last; v0 += width) {
    const int c = (v0 + tv) * V;
    const bool on = team < teams && v0 + tv < last;
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
    if (team == 0 && on) {
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

// A gradient in planes for a table of at most kPrivRows rows needs no sort and
// no turning: a block owns up to 4 * kPrivWarps columns of a table of its own
// in shared memory and a split of the items, a warp four of the columns.  The
// warp adds 32 items at a time in order: lanes with the same id first sum
// their values by pointer jumping along the lanes (log2 of the largest
// group's steps, none if all ids differ), then each group's first lane adds
// to the table.  The groups are found once for all columns.  g is read once,
// as it lies; the splits' tables are summed by k_join_tables in order.
// Bound by instruction issue and the shared memory's latency: 2.5M x 48 for
// 1024 rows take 241 us against 358 by the sort, 150K x 12 take 21 against 37.
// Against the number of rows, in us, private tables / sort:
//   2.5M x     512 rows   1024       1536       2048       4096
//     3        67/101     67/113     71/113     88/113     124/111
//    12        70/155     82/168    124/168    124/168     334/167
//    27       121/239    164/252    240/251    325/251     726/253
//    48       172/346    241/358    310/358    420/358    1155/359
// (150K items cross a little later.)  More rows leave a block fewer
// columns, and g's ids are read again for each.  Up to 1024 rows the form wins
// by a third or more at every width; up to 2048 by less and at some widths
// only, and those tables take the sort.  For a gradient in rows the sort is
// faster at any size (300K x 128 for 1000 rows: 64 us; private tables took
// 157).
constexpr int kPrivRows = 1024, kPrivWarps = 8, kPrivTile = 256, kPrivBytes = 96 * 1024;

struct PrivShape {
  int warps, cols, col_groups;  // columns per block
  int64_t splits, per;          // items per split
  size_t smem, partial;         // bytes
  bool use;
  PrivShape(int64_t n, int64_t rows, int all, bool planes)
      : use(planes && n > kSmallItems && rows <= kPrivRows) {
    if (!use) return;
    int64_t c = kPrivBytes / (4 * rows) / 4 * 4;
    if (c > 4 * kPrivWarps) c = 4 * kPrivWarps;
    col_groups = (int)((all + c - 1) / c);
    cols = ((all + col_groups - 1) / col_groups + 3) / 4 * 4;
    col_groups = (all + cols - 1) / cols;
    warps = cols / 4;
    smem = (size_t)rows * cols * 4;
    // blocks for the device, of two tiles or more, whose tables are at most as
    // large as the items or stay in L2
    int64_t at_once = (int64_t)(220 * 1024 / (smem + 6 * 1024));
    if (at_once > 8) at_once = 8;
    splits = 148 * at_once / col_groups;
    const int64_t table = rows * all * 4, most = n / rows > (16 << 20) / table ? n / rows : (16 << 20) / table;
    if (splits > most) splits = most;
    if (splits > n / (2 * kPrivTile)) splits = n / (2 * kPrivTile);
    if (splits < 1) splits = 1;
    per = ((n + splits - 1) / splits + kPrivTile - 1) / kPrivTile * kPrivTile;
    splits = (n + per - 1) / per;
    partial = (size_t)splits * ((all + 3) / 4) * rows * 16;
  }
};

template <class T>
__global__ void __launch_bounds__(32 * kPrivWarps)
k_private_sums(const T* __restrict__ g, int64_t cs, int all,
               const __grid_constant__ Ids src, int64_t n, int64_t per, int64_t splits, int cols,
               float* __restrict__ partial, int32_t* dev_status) {
  constexpr int GROUPS = kPrivTile / 32;
  extern __shared__ __align__(16) float s_table[];  // [warp][rows][4]
  __shared__ int32_t s_id[2][kPrivTile];
  __shared__ uint32_t s_mask[2][kPrivTile];
  __shared__ int s_steps[2][GROUPS];
  wait_for_prior_grids();
  const int t = threadIdx.x, lane = t & 31, w = t >> 5, threads = blockDim.x;
  const int rows = (int)src.rows;
  const int64_t split = blockIdx.x % splits;
  const int c0 = (int)(blockIdx.x / splits) * cols + 4 * w;  // this warp's first column
  const int64_t first = split * per, last = min(first + per, n);
  for (int i = t; i < cols / 4 * rows; i += threads)
    reinterpret_cast<float4*>(s_table)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float4* table = reinterpret_cast<float4*>(s_table) + w * rows;
  const uint32_t below = (1u << lane) - 1;
  int buf = 0;
  const T* col[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) col[i] = g + (int64_t)min(c0 + i, all - 1) * cs;
  // the ids of a tile are fetched while the tile before is summed
  int32_t ids[GROUPS];
  const auto fetch_ids = [&](int64_t j0) {
#pragma unroll
    for (int q = 0; q < GROUPS; ++q) {
      const int64_t j = j0 + t + q * threads;
      ids[q] = t + q * threads < kPrivTile && j < last
                   ? id_of(src.ids, src.n_ids, src.index, j, src.rows, dev_status)
                   : -1;
    }
  };
  fetch_ids(first);
  for (int64_t j0 = first; j0 < last; j0 += kPrivTile, buf ^= 1) {
#pragma unroll
    for (int q = 0; q < GROUPS; ++q) {
      const int i = t + q * threads;
      if (i >= kPrivTile) break;  // whole warps: threads and the tile are multiples of 32
      const uint32_t same = __match_any_sync(0xffffffffu, ids[q]);
      const uint32_t mask = ids[q] >= 0 ? same : 1u << lane;
      const int most = __reduce_max_sync(0xffffffffu, __popc(mask));
      s_id[buf][i] = ids[q];
      s_mask[buf][i] = mask;
      if (lane == 0) s_steps[buf][i >> 5] = 32 - __clz(most - 1);  // ceil(log2(most))
    }
    // rows and columns that do not exist are read at the last ones and not used
    Pack<T, 4> x[GROUPS];
    const auto fetch_rows = [&](auto at) {  // at(k): item of this lane in group k
#pragma unroll
      for (int k = 0; k < GROUPS; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[k].x[i] = __ldcs(col[i] + at(k));
      }
    };
    if (j0 + kPrivTile <= last) fetch_rows([&](int k) { return j0 + lane + k * 32; });
    else fetch_rows([&](int k) { return min(j0 + lane + k * 32, last - 1); });
    if (j0 + kPrivTile < last) fetch_ids(j0 + kPrivTile);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      const int32_t id = s_id[buf][k * 32 + lane];
      const uint32_t mask = s_mask[buf][k * 32 + lane];
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = to_f(x[k].x[i]);
      int steps = s_steps[buf][k];
      if (steps > 0) {
        const uint32_t above = mask & ~below & ~(1u << lane);
        int next = above ? __ffs(above) - 1 : 32;  // the group's next lane; 32: none
        do {
          const int from = next & 31, jump = __shfl_sync(0xffffffffu, next, from);
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = __shfl_sync(0xffffffffu, v[i], from);
          if (next < 32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += y[i];
            next = jump;
          }
        } while (--steps > 0);
      }
      if (id >= 0 && !(mask & below)) {
        float4 y = table[id];
        y.x += v[0], y.y += v[1], y.z += v[2], y.w += v[3];
        table[id] = y;
      }
      __syncwarp();
    }
  }
  __syncthreads();
  // partial[split][four columns][row][4], as the table lies
  const int quads = (all + 3) / 4, from = (int)(blockIdx.x / splits) * (cols / 4);
  const int size = min(cols / 4, quads - from) * rows;
  float4* o = reinterpret_cast<float4*>(partial) + (split * quads + from) * rows;
  for (int i = t; i < size; i += threads) o[i] = reinterpret_cast<const float4*>(s_table)[i];
}

// dtable[k][c] (+)= scale * sum of the splits' tables: a thread sums four
// columns of a row over one of eight stretches of the splits, sixteen loads in
// flight, and the stretches are joined in order.
__global__ void __launch_bounds__(kThreads)
k_join_tables(const float4* __restrict__ partial, int64_t splits, int cols, int rows, float scale,
              float* __restrict__ dtable, int64_t ld, bool accumulate) {
  constexpr int PARTS = kThreads / 32;
  __shared__ float4 s_sum[PARTS][32];
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t total = (int64_t)((cols + 3) / 4) * rows, e = (int64_t)blockIdx.x * 32 + lane;
  const int64_t each = (splits + PARTS - 1) / PARTS, a = w * each, b = min(a + each, splits);
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto add = [&](const float4& x) { sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w; };
  if (e < total) {
    const float4* p = partial + e;
#pragma unroll 16
    for (int64_t i = a; i < b; ++i) add(p[i * total]);
  }
  s_sum[w][lane] = sum;
  __syncthreads();
  if (w == 0 && e < total) {
    for (int k = 1; k < PARTS; ++k) add(s_sum[k][lane]);
    const int c = (int)(e / rows) * 4;
    float* d = dtable + e % rows * ld + c;
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < cols) d[i] = accumulate ? d[i] + scale * v[i] : scale * v[i];
  }
}

unsigned blocks_for(int64_t threads) { return (unsigned)((threads + kThreads - 1) / kThreads); }

int key_bits(int64_t rows) { return rows > 1 ? 64 - __builtin_clzll((unsigned long long)(rows - 1)) : 0; }

struct LookupWs {
  float* partial;   // private tables
  uint2* pairs[2];  // the sorted order ends in pairs[0]
  uint32_t* counts;
  uint32_t* total;
  uint32_t* pkey[2];
  float* psum[2];
  uint4* rows;  // the items' rows, for a gradient in planes
  int ldp;
  size_t bytes;
};

struct Passes {
  int count, bits;
  explicit Passes(int64_t rows) {
    const int all = key_bits(rows);
    count = all <= kMaxDigit ? 1 : (all + kMaxDigit - 1) / kMaxDigit;
    bits = (all + count - 1) / count;
  }
};

LookupWs carve_lookup(void* ws, size_t cap, int64_t n, int64_t rows, int cols, int planes_es) {
  LookupWs w{};
  if (n <= kSmallItems) return w;
  Carver cv(ws, cap);
  w.ldp = (cols + 7) / 8 * 8;
  const Passes ps(rows);
  w.pairs[0] = cv.take<uint2>(n);
  w.pairs[1] = cv.take<uint2>(n);
  const int64_t tiles = (n + kSortTile - 1) / kSortTile;
  w.counts = cv.take<uint32_t>(((size_t)1 << ps.bits) * tiles * (tiles <= kFewTiles ? ps.count : 1));
  w.total = cv.take<uint32_t>((size_t)1 << ps.bits);
  // partials: the most that any type and alignment leaves
  int64_t m = n;
  for (int k = 0; k < 2; ++k) {
    int64_t most = k ? RunShape(m, cols, 4, 4, false).blocks : 0;
    for (int es = 2; !k && es <= 4; es += 2)
      for (int V = 1; V <= 16 / es; V += 16 / es - 1) {
        const int64_t b = RunShape(m, cols, V, es, true).blocks;
        if (b > most) most = b;
      }
    m = 2 * most;
    w.pkey[k] = cv.take<uint32_t>(m);
    w.psum[k] = cv.take<float>((size_t)m * w.ldp);
  }
  // behind what a kept order needs
  const PrivShape priv(n, rows, cols, planes_es != 0);
  if (priv.use) w.partial = cv.take<float>(priv.partial / 4);
  else if (planes_es) w.rows = cv.take<uint4>((size_t)n * (((size_t)cols * planes_es + 15) / 16));
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

constexpr int kMaxCols = 1 << 30;  // columns are counted in int, rounded up

gs_status check_ids(const int32_t* ids, int64_t n_ids, const int32_t* index, int64_t n) {
  if (n < 0 || n_ids < 0) return GS_ERR_ARG;
  if (n > (int64_t)INT32_MAX) return GS_ERR_UNSUPPORTED;  // positions are int32
  if (n > 0 && ((!ids && n_ids > 0) || (!index && n_ids < n))) return GS_ERR_ARG;
  if (!aligned(ids, 4) || !aligned(index, 4)) return GS_ERR_ARG;
  return GS_OK;
}

// Sorts the items by id into w.pairs[0]; also clears `zeros` floats at dtable.
gs_status plan_lookup(const int32_t* ids, int64_t n_ids, const int32_t* index, int64_t n,
                      int64_t rows, const LookupWs& w, float* dtable, int64_t zeros,
                      int32_t* dev_status, cudaStream_t s) {
  const Passes ps(rows);
  const Ids src{ids, index, n_ids, rows};
  const unsigned tiles = (unsigned)((n + kSortTile - 1) / kSortTile);
  const bool few = tiles <= kFewTiles;
  uint32_t* counts = w.counts;
  for (int p = 0; p < ps.count; ++p) {
    uint2* from = w.pairs[(ps.count - p) & 1];
    uint2* to = w.pairs[(ps.count - 1 - p) & 1];
    const int shift = p * ps.bits;
    if (p == 0 || !few) {
      GS_TRY(launch_dependent(p == 0 ? k_sort_count<true> : k_sort_count<false>, tiles, kThreads, 0, s,
                              src, from, n, shift, ps.bits, counts, few, few ? ps.count - 1 : 0,
                              dtable, zeros, dev_status));
      GS_LAUNCH_CHECK();
    }
    uint32_t* next = few && p + 1 < ps.count ? counts + ((size_t)tiles << ps.bits) : nullptr;
    if (!few) {
      GS_TRY(launch_dependent(k_sort_scan, 1u << ps.bits, kThreads, 0, s, counts, tiles, w.total));
      GS_LAUNCH_CHECK();
    }
    GS_TRY(launch_dependent(few ? k_sort_scatter<true> : k_sort_scatter<false>, tiles, kThreads,
                            scatter_smem(ps.bits), s, from, n, shift, ps.bits, counts, w.total, next,
                            to));
    GS_LAUNCH_CHECK();
    if (next) counts = next;
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

template <class T, int V, bool FIRST>
gs_status launch_sums(const uint2* pairs, const uint32_t* keys, int64_t n, const RunShape& sh,
                      const T* g, int64_t rs, int cols, float scale, const gs_matrix* dtable,
                      bool accumulate, uint32_t* pkey, float* psum, int ldp, int32_t* dev_status,
                      cudaStream_t s) {
  if (sh.blocks * sh.col_tiles > (int64_t)INT32_MAX) return GS_ERR_UNSUPPORTED;
  static std::atomic<unsigned long long> once{0};
  GS_TRY(smem_attrs_once((const void*)k_run_sums<T, V, FIRST>,
                         kRunRowBytes + 2 * kThreads * V * 4 + kRunEntries * 8, &once));
  GS_TRY(launch_dependent(k_run_sums<T, V, FIRST>, (unsigned)(sh.blocks * sh.col_tiles), kThreads,
                          sh.smem, s, pairs, keys, n, sh, g, rs, cols, scale,
                          static_cast<float*>(dtable->data), dtable->row_stride,
                          (uint32_t)dtable->rows,
                          vector_of(dtable->data, dtable->row_stride, cols, 4, 4) == 4, accumulate,
                          pkey, psum, ldp, dev_status));
  GS_LAUNCH_CHECK();
  return GS_OK;
}

template <class T, int V>
gs_status run_sums(const T* g, int64_t rs, int64_t n, int cols, float scale, const gs_matrix* dtable,
                   bool accumulate, const LookupWs& w, int32_t* dev_status, cudaStream_t s) {
  RunShape sh(n, cols, V, sizeof(T), true);
  gs_status st = launch_sums<T, V, true>(w.pairs[0], nullptr, n, sh, g, rs, cols, scale, dtable,
                                         accumulate, w.pkey[0], w.psum[0], w.ldp, dev_status, s);
  for (int from = 0; st == GS_OK && sh.blocks > 1; from ^= 1) {
    const int64_t m = 2 * sh.blocks;
    sh = RunShape(m, cols, 4, 4, false);
    st = launch_sums<float, 4, false>(nullptr, w.pkey[from], m, sh, w.psum[from], w.ldp, cols, scale,
                                      dtable, accumulate, w.pkey[from ^ 1], w.psum[from ^ 1], w.ldp,
                                      dev_status, s);
  }
  return st;
}

template <class TT, class TO, int V>
gs_status launch_rows(const gs_matrix* t, const int32_t* ids, int64_t n_ids, const int32_t* index,
                      float scale, const gs_matrix* o, int32_t* dev_status, cudaStream_t s) {
  const int nv = o->cols / V;
  int items = kThreads * kRowIlp / nv;
  if (items < 1) items = 1;
  const int64_t blocks = (o->rows + items - 1) / items;
  GS_TRY(launch_dependent(k_lookup_rows<TT, TO, V>, (unsigned)blocks, kThreads, 0, s,
                          static_cast<const TT*>(t->data), t->row_stride, t->rows, ids, n_ids, index,
                          scale, static_cast<TO*>(o->data), o->rows, o->row_stride,
                          Div((uint32_t)nv), items, dev_status));
  GS_LAUNCH_CHECK();
  return GS_OK;
}

template <class TT, class TO>
gs_status lookup_by(const gs_matrix* t, const int32_t* ids, int64_t n_ids, const int32_t* index,
                    float scale, const gs_matrix* o, int32_t* dev_status, cudaStream_t s) {
  if (o->col_stride != 1) {
    constexpr int V = 16 / sizeof(TT);
    const int cols = o->cols;
    const int64_t words = ((int64_t)cols * sizeof(TT) + 3) / 4;
    const int al = vector_of(t->data, t->row_stride, cols, sizeof(TT), 2 * V);
    const unsigned blocks = blocks_for(o->rows);
    if (al >= V && words > 16) {
      static std::atomic<unsigned long long> once{0};
      GS_TRY(smem_attrs_once((const void*)k_lookup_planes_staged<TT, TO>, (int)kStageSmem, &once));
      GS_TRY(launch_dependent(k_lookup_planes_staged<TT, TO>, blocks, kThreads, kStageSmem, s,
                              static_cast<const TT*>(t->data), t->row_stride, t->rows, cols, ids,
                              n_ids, index, scale, static_cast<TO*>(o->data), o->rows,
                              o->col_stride, dev_status));
      GS_LAUNCH_CHECK();
      return GS_OK;
    }
#define GS_LOOKUP_PLANES(NW, AL)                                                                  \
  GS_TRY(launch_dependent(k_lookup_planes<TT, TO, NW, AL>, blocks, kThreads, 0, s,                 \
                          static_cast<const TT*>(t->data), t->row_stride, t->rows, cols, ids,      \
                          n_ids, index, scale, static_cast<TO*>(o->data), o->rows, o->col_stride, \
                          dev_status))
    if (words <= 16) {
      if (al == 2 * V) GS_LOOKUP_PLANES(16, 32);
      else if (al == V) GS_LOOKUP_PLANES(16, 16);
      else GS_LOOKUP_PLANES(16, 0);
    } else {
      GS_LOOKUP_PLANES(48, 0);  // aligned rows of that size went above
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
  if (table->cols > kMaxCols) return GS_ERR_UNSUPPORTED;
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
  if (n < 0 || n > (int64_t)INT32_MAX || rows < 1 || rows > (int64_t)INT32_MAX || cols < 1 ||
      cols > kMaxCols)
    return 0;
  const size_t b = carve_lookup(nullptr, 0, n, rows, cols, planes ? 4 : 0).bytes;
  return b > 256 ? b : 256;
}

extern "C" gs_status gs_lookup_plan(const int32_t* ids, int64_t n_ids, const int32_t* index,
                                    int64_t n, int64_t rows, int32_t cols, void* ws, size_t ws_bytes,
                                    int32_t* dev_status, gs_stream stream) {
  const gs_status st = check_ids(ids, n_ids, index, n);
  if (st != GS_OK) return st;
  if (rows < 1 || rows > (int64_t)INT32_MAX || cols < 1) return GS_ERR_ARG;
  if (cols > kMaxCols) return GS_ERR_UNSUPPORTED;
  if (n == 0) return GS_OK;
  const LookupWs w = carve_lookup(ws, ws_bytes, n, rows, cols, 0);
  if (!ws || w.bytes > ws_bytes || ws_bytes < 256) return GS_ERR_CAPACITY;
  if (!aligned(ws, 256)) return GS_ERR_ARG;
  if (!w.pairs[0]) return GS_OK;  // such gradients need no order
  return plan_lookup(ids, n_ids, index, n, rows, w, nullptr, 0, dev_status, to_stream(stream));
}

namespace gs {
namespace {

template <class T, int V>
gs_status small_grad(const gs_matrix* g, const int32_t* ids, int64_t n_ids, const int32_t* index,
                     float scale, const gs_matrix* dtable, bool accumulate, int32_t* dev_status,
                     cudaStream_t s) {
  // a row per block while that leaves at most four blocks for each SM, and
  // the columns cut where the rows do not fill the device
  const int64_t rows = dtable->rows;
  int64_t blocks = rows < 148 * 4 ? rows : 148 * 4;
  int64_t per = (rows + blocks - 1) / blocks;
  if (per > kSmallRows) per = kSmallRows;
  blocks = (rows + per - 1) / per;
  const int nv = (g->cols + V - 1) / V;
  int64_t col_tiles = 148 / blocks;
  if (col_tiles > nv) col_tiles = nv;
  if (col_tiles < 1) col_tiles = 1;
  const int share = (int)((nv + col_tiles - 1) / col_tiles);
  col_tiles = (nv + share - 1) / share;
  GS_TRY(launch_dependent(k_small_grad<T, V>, (unsigned)(blocks * col_tiles), kThreads, 0, s,
                          static_cast<const T*>(g->data), g->row_stride, g->col_stride, g->cols,
                          share, (unsigned)col_tiles, ids, n_ids, index, (int)g->rows, scale,
                          static_cast<float*>(dtable->data), dtable->row_stride, rows, (int)per,
                          accumulate, dev_status));
  GS_LAUNCH_CHECK();
  return GS_OK;
}

template <class T>
gs_status private_grad(const gs_matrix* g, const Ids& src, float scale, const gs_matrix* dtable,
                       bool accumulate, const PrivShape& ps, float* partial, int32_t* dev_status,
                       cudaStream_t s) {
  const int64_t join = (((int64_t)g->cols + 3) / 4 * src.rows + 31) / 32;
  if (join > (int64_t)INT32_MAX || ps.splits * ps.col_groups > (int64_t)INT32_MAX)
    return GS_ERR_UNSUPPORTED;
  static std::atomic<unsigned long long> once{0};
  GS_TRY(smem_attrs_once((const void*)k_private_sums<T>, kPrivBytes, &once));
  GS_TRY(launch_dependent(k_private_sums<T>, (unsigned)(ps.splits * ps.col_groups), 32 * ps.warps,
                          ps.smem, s, static_cast<const T*>(g->data), g->col_stride, g->cols, src,
                          g->rows, ps.per, ps.splits, ps.cols, partial, dev_status));
  GS_LAUNCH_CHECK();
  const int rows = (int)src.rows;
  GS_TRY(launch_dependent(k_join_tables, (unsigned)join, kThreads, 0, s,
                          reinterpret_cast<const float4*>(partial), ps.splits, g->cols, rows, scale,
                          static_cast<float*>(dtable->data), dtable->row_stride, accumulate));
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
  const PrivShape ps(n, dtable->rows, cols, planes);
  if (ps.use)
    return private_grad<T>(g, Ids{ids, index, n_ids, dtable->rows}, scale, dtable, accumulate, ps,
                           w.partial, dev_status, s);
  if (planes) {
    const int vecs = (cols + V - 1) / V;
    static std::atomic<unsigned long long> once{0};
    GS_TRY(smem_attrs_once((const void*)k_planes_to_rows<T>, (int)Turn<T>::kSmem, &once));
    GS_TRY(launch_dependent(k_planes_to_rows<T>, (unsigned)((n + kTurnItems - 1) / kTurnItems),
                            kThreads, Turn<T>::smem(vecs), s, data, g->col_stride, cols, n, w.rows,
                            vecs));
    GS_LAUNCH_CHECK();
    return run_sums<T, V>(reinterpret_cast<const T*>(w.rows), (int64_t)vecs * V, n, cols, scale,
                          dtable, accumulate, w, dev_status, s);
  }
  return vec ? run_sums<T, V>(data, g->row_stride, n, cols, scale, dtable, accumulate, w,
                              dev_status, s)
             : run_sums<T, 1>(data, g->row_stride, n, cols, scale, dtable, accumulate, w,
                              dev_status, s);
}

}  // namespace
}  // namespace gs

extern "C" gs_status gs_lookup_bwd(const gs_matrix* g, const int32_t* ids, int64_t n_ids,
                                   const int32_t* index, double scale, const gs_matrix* dtable,
                                   uint32_t flags, void* ws, size_t ws_bytes, int32_t* dev_status,
                                   gs_stream stream) {
  if (flags & ~(GS_LOOKUP_ACCUMULATE | GS_LOOKUP_PLANNED)) return GS_ERR_ARG;
  if (!isfinite((float)scale)) return GS_ERR_ARG;  // times a sum of 0: NaN in rows that nothing uses
  if (!good_matrix(g) || !good_matrix(dtable) || g->cols != dtable->cols) return GS_ERR_ARG;
  if (dtable->rows < 1 || dtable->rows > (int64_t)INT32_MAX) return GS_ERR_ARG;
  if (dtable->dtype != GS_F32 || dtable->col_stride != 1 || g->cols > kMaxCols)
    return GS_ERR_UNSUPPORTED;
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
  const bool sorted = n > kSmallItems && !PrivShape(n, rows, g->cols, planes_es != 0).use;
  const bool plan = !(flags & GS_LOOKUP_PLANNED) && sorted;
  float* dt = static_cast<float*>(dtable->data);
  // rows that no item uses: cleared by the sort's first kernel where the table
  // is contiguous and no block of it gets more than 256 KB to clear
  const int64_t elements = rows * dtable->cols, tiles = (n + kSortTile - 1) / kSortTile;
  const bool fused = plan && !accumulate && dtable->row_stride == dtable->cols &&
                     aligned(dt, 16) && elements <= tiles * 65536;
  if (!accumulate && !fused && (n == 0 || sorted) &&
      cudaMemset2DAsync(dt, dtable->row_stride * 4, 0, (size_t)g->cols * 4, rows, s) != cudaSuccess) {
    (void)cudaGetLastError();  // leave no error for the next call
    return GS_ERR_CUDA;
  }
  if (n == 0) return GS_OK;
  if (plan) {
    const gs_status ps = plan_lookup(ids, n_ids, index, n, rows, w, dt, fused ? elements : 0,
                                     dev_status, s);
    if (ps != GS_OK) return ps;
  }
  const float sc = (float)scale;
  switch (g->dtype) {
    case GS_F32: return lookup_grad<float>(g, ids, n_ids, index, sc, dtable, accumulate, w, dev_status, s);
    case GS_F16: return lookup_grad<__half>(g, ids, n_ids, index, sc, dtable, accumulate, w, dev_status, s);
    default: return lookup_grad<__nv_bfloat16>(g, ids, n_ids, index, sc, dtable, accumulate, w, dev_status, s);
  }
}
