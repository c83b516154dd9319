// Embedding lookup straight from a gathered flat buffer, and its gradient
// straight into the packed flat buffer, on gfx950: kernels and the
// rs_embed_rows / rs_embed_grad / rs_embed_workspace entry points. They are
// the unpack and pack of one tensor ("veScale-FSDP: flexible, structure-aware
// sharding at 10K-GPU scale", feynmanwiki walkthrough, DBuffer paragraphs: a
// tensor is its planned slice, and group-fused scale / add / zero before the
// reduction) for the rows that a batch of tokens names, instead of a copy of
// the whole table and a dense gradient.
//
//   lookup:    out[t] = scale * table[ids[t]]
//   gradient:  packed[r] = [prev[r] +] sigma * sum over t with ids[t] = r of dy[t]
//
// Both move bytes only. The gradient sums in a fixed order without atomics:
// the tokens are sorted by (row, token); whole chunks of 64 sorted tokens of
// one row (common tokens) are summed by workgroups of their own; then each row
// adds its chunk sums and its remaining tokens in order.
#include "host_common.h"

namespace rs {
namespace {

constexpr uint32_t kNoRow = 0xffffffffu;   // sorts behind every row

// Row of token t, kNoRow where the id names none.
__device__ __forceinline__ uint32_t row_of(const void* ids, bool wide, int64_t t, uint32_t rows) {
  if (wide) {
    const int64_t v = static_cast<const int64_t*>(ids)[t];
    return v >= 0 && v < static_cast<int64_t>(rows) ? static_cast<uint32_t>(v) : kNoRow;
  }
  const int32_t v = static_cast<const int32_t*>(ids)[t];
  return v >= 0 && static_cast<uint32_t>(v) < rows ? static_cast<uint32_t>(v) : kNoRow;
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  if constexpr (BF16) {
    In<true>::widen(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at), x);
  } else {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) { x[e] = a[e]; x[4 + e] = b[e]; }
  }
}

// ------------------------------------------------------------------ lookup

constexpr int kLookVecs = 4;   // vectors (or elements) per thread

// Work is numbered over tokens * units of a row: a unit is 8 elements (VEC),
// or one element where the width is no multiple of 8. 32-bit arithmetic after
// the workgroup's own first token.
template <bool IN16, bool OUT16, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_rows_kernel(const void* table, const void* ids, bool wide,
                                                              int64_t n_units, uint32_t units, uint32_t rows,
                                                              int64_t cols, float scale, void* out) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kLookVecs);
  const int64_t t0 = first / units;
  const uint32_t u0 = static_cast<uint32_t>(first - t0 * units);
#pragma unroll
  for (int k = 0; k < kLookVecs; ++k) {
    const uint32_t w = k * kThreads + threadIdx.x;
    if (first + w >= n_units) break;
    const uint32_t x = u0 + w, d = x / units, u = x - d * units;
    const int64_t t = t0 + d;
    const uint32_t r = row_of(ids, wide, t, rows);
    if constexpr (VEC) {
      float v[8] = {};
      if (r != kNoRow) {
        load8<IN16>(table, static_cast<int64_t>(r) * cols + u * 8, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], scale);
      }
      if constexpr (OUT16) {
        uint32_t b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = bf16_rne(v[e]);
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + t * cols + u * 8) =
            u32x4{b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16};
      } else {
        f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(out) + t * cols + u * 8);
        o[0] = f32x4{v[0], v[1], v[2], v[3]};
        o[1] = f32x4{v[4], v[5], v[6], v[7]};
      }
    } else {
      const float v = r == kNoRow ? 0.0f : __fmul_rn(In<IN16>::elem(table, static_cast<int64_t>(r) * cols + u), scale);
      if constexpr (OUT16) static_cast<uint16_t*>(out)[t * cols + u] = static_cast<uint16_t>(bf16_rne(v));
      else static_cast<float*>(out)[t * cols + u] = v;
    }
  }
}

// ------------------------------------------------------------------ sort

constexpr int kRun = 2048;            // keys sorted in LDS by one workgroup
constexpr int kSortThreads = 1024;
constexpr int kSumChunk = 64;         // sorted tokens of one row summed ahead

// Keys (row << 32 | token) of kRun tokens, sorted in LDS by a bitonic network
// (every key differs, so the order is unique); n is the power of two that
// holds the largest run. A single run goes out as the sorted rows and tokens.
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(const void* ids, bool wide, int64_t n_ids,
                                                                  uint32_t rows, int n, uint64_t* keys, uint32_t* srow,
                                                                  uint32_t* stok) {
  __shared__ uint64_t s[kRun];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kRun;
  for (int i = threadIdx.x; i < n; i += kSortThreads) {
    const int64_t t = base + i;
    s[i] = t < n_ids ? static_cast<uint64_t>(row_of(ids, wide, t, rows)) << 32 | static_cast<uint32_t>(t) : ~0ull;
  }
  for (int size = 2; size <= n; size *= 2) {
    for (int step = size / 2; step > 0; step /= 2) {
      __syncthreads();
      for (int p = threadIdx.x; p < n / 2; p += kSortThreads) {
        const int i = 2 * p - (p & (step - 1)), j = i + step;
        const uint64_t a = s[i], b = s[j];
        if ((a > b) == ((i & size) == 0)) {
          s[i] = b;
          s[j] = a;
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n && base + i < n_ids; i += kSortThreads) {
    if (keys) {
      keys[base + i] = s[i];
    } else {
      srow[i] = static_cast<uint32_t>(s[i] >> 32);
      stok[i] = static_cast<uint32_t>(s[i]);
    }
  }
}

// Sorted runs -> one sorted list: a key's place is its place in its own run
// plus the number of smaller keys in every other run, found by binary search,
// eight runs at a time so that their loads overlap.
__global__ __launch_bounds__(kThreads) void embed_merge_kernel(const uint64_t* __restrict__ keys, int64_t n_ids,
                                                               uint32_t* srow, uint32_t* stok) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= n_ids) return;
  const uint64_t key = keys[i];
  const int64_t own = i / kRun, runs = (n_ids + kRun - 1) / kRun;
  int64_t place = i - own * kRun;
  constexpr int kAt = 8;
  for (int64_t r0 = 0; r0 < runs; r0 += kAt) {
    int lo[kAt], len[kAt];   // smaller keys lie in [0, lo), the undecided ones in [lo, lo + len)
#pragma unroll
    for (int r = 0; r < kAt; ++r) {
      lo[r] = 0;
      const int64_t at = (r0 + r) * kRun;
      len[r] = r0 + r == own || at >= n_ids ? 0 : static_cast<int>(n_ids - at < kRun ? n_ids - at : kRun);
    }
    for (int step = 0; step < 12; ++step) {   // 2^11 = kRun: twelve halvings leave nothing undecided
#pragma unroll
      for (int r = 0; r < kAt; ++r) {
        if (len[r] > 0) {
          const int half = len[r] / 2;
          if (keys[(r0 + r) * kRun + lo[r] + half] < key) {
            lo[r] += half + 1;
            len[r] -= half + 1;
          } else {
            len[r] = half;
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kAt; ++r) place += lo[r];
  }
  srow[place] = static_cast<uint32_t>(key >> 32);
  stok[place] = static_cast<uint32_t>(key);
}

// ------------------------------------------------------------------ gradient

// Columns of one wave: lane l holds four. Whole vectors of four neighbours
// where the width is a multiple of 4, else single columns 64 apart.
constexpr int kWaveCols = 4 * kWave;

template <bool VEC>
__device__ __forceinline__ int64_t col_of(int64_t c0, int lane, int e) {
  return VEC ? c0 + lane * 4 + e : c0 + e * kWave + lane;
}

template <bool BF16, bool VEC>
__device__ __forceinline__ f32x4 load_cols(const void* p, int64_t row_at, int64_t c0, int64_t cols, int lane) {
  f32x4 x = {};
  if constexpr (VEC) {
    const int64_t c = c0 + lane * 4;
    if (c < cols) {
      if constexpr (BF16) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + row_at + c);
        x = f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                  __uint_as_float(w.y & 0xffff0000u)};
      } else {
        x = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + row_at + c);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t c = col_of<false>(c0, lane, e);
      if (c < cols) x[e] = In<BF16>::elem(p, row_at + c);
    }
  }
  return x;
}

// A 64-token window of the sorted list in a wave's registers: lane l holds
// position base + l.
struct Window {
  int64_t base = -1;
  uint32_t row = kNoRow, tok = 0;
  __device__ __forceinline__ void at(int64_t pos, const uint32_t* srow, const uint32_t* stok, int64_t n, int lane) {
    const int64_t b = pos & ~static_cast<int64_t>(kSumChunk - 1);
    if (b == base) return;
    base = b;
    row = b + lane < n ? srow[b + lane] : kNoRow;
    tok = b + lane < n ? stok[b + lane] : 0u;
  }
};

// Sum of tokens [from, to) of the window for this wave's columns, in order.
template <bool BF16, bool VEC>
__device__ __forceinline__ f32x4 sum_tokens(f32x4 sum, const Window& w, int from, int to, const void* dy, int64_t c0,
                                            int64_t cols, int lane) {
  int i = from;
  for (; i + 4 <= to; i += 4) {   // four rows on their way at a time
    f32x4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t t = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(w.tok), i + k));
      x[k] = load_cols<BF16, VEC>(dy, static_cast<int64_t>(t) * cols, c0, cols, lane);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sum += x[k];
  }
  for (; i < to; ++i) {
    const uint32_t t = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(w.tok), i));
    sum += load_cols<BF16, VEC>(dy, static_cast<int64_t>(t) * cols, c0, cols, lane);
  }
  return sum;
}

// Chunks of kSumChunk sorted tokens that are all one row's -> their sums.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_chunk_kernel(const uint32_t* __restrict__ srow,
                                                               const uint32_t* __restrict__ stok, int64_t n_ids,
                                                               const void* dy, int64_t cols, float* part) {
  const int lane = threadIdx.x % kWave;
  const int64_t chunk = blockIdx.x;
  Window w;
  w.at(chunk * kSumChunk, srow, stok, n_ids, lane);
  const uint32_t first = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(w.row)));
  if (first == kNoRow || !__all(w.row == first)) return;
  const int64_t c0 = (static_cast<int64_t>(blockIdx.y) * (kThreads / kWave) + threadIdx.x / kWave) * kWaveCols;
  if (c0 >= cols) return;
  const f32x4 sum = sum_tokens<BF16, VEC>(f32x4{}, w, 0, kSumChunk, dy, c0, cols, lane);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t c = col_of<VEC>(c0, lane, e);
    if (c < cols) part[chunk * cols + c] = sum[e];
  }
}

// Sum over the tokens of row r from sorted position pos on; moves pos past them.
template <bool BF16, bool VEC>
__device__ __forceinline__ f32x4 sum_row(uint32_t r, int64_t& pos, Window& w, const uint32_t* srow,
                                         const uint32_t* stok, int64_t n_ids, const void* dy, const float* part,
                                         int64_t c0, int64_t cols, int lane) {
  f32x4 sum = {};
  while (pos < n_ids) {
    w.at(pos, srow, stok, n_ids, lane);
    const int from = static_cast<int>(pos - w.base);
    const int count = __popcll(__ballot(w.row == r && lane >= from));   // a row's positions are neighbours
    if (count == 0) break;
    if (part && count == kSumChunk)
      sum += load_cols<false, VEC>(part, w.base / kSumChunk * cols, c0, cols, lane);
    else
      sum = sum_tokens<BF16, VEC>(sum, w, from, from + count, dy, c0, cols, lane);
    pos += count;
    if (from + count < kSumChunk) break;   // the row ends inside the window
  }
  return sum;
}

template <bool OUT16, bool VEC>
__device__ __forceinline__ void store_row(void* packed, const float* prev, int64_t row_at, f32x4 sum, float sigma,
                                          int64_t c0, int64_t cols, int lane) {
  f32x4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = __fmul_rn(sum[e], sigma);
  if (prev) {
    const f32x4 p = load_cols<false, VEC>(prev, row_at, c0, cols, lane);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __fadd_rn(p[e], y[e]);
  }
  if constexpr (VEC) {
    const int64_t c = c0 + lane * 4;
    if (c < cols) {
      if constexpr (OUT16)
        stg(reinterpret_cast<u32x2*>(static_cast<uint16_t*>(packed) + row_at + c),
            u32x2{bf16_rne(y[0]) | bf16_rne(y[1]) << 16, bf16_rne(y[2]) | bf16_rne(y[3]) << 16});
      else
        stg(reinterpret_cast<f32x4*>(static_cast<float*>(packed) + row_at + c), y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t c = col_of<false>(c0, lane, e);
      if (c < cols) {
        if constexpr (OUT16) static_cast<uint16_t*>(packed)[row_at + c] = static_cast<uint16_t>(bf16_rne(y[e]));
        else static_cast<float*>(packed)[row_at + c] = y[e];
      }
    }
  }
}

// First sorted position whose row is at least r: every lane probes, so a step
// divides what is left by 64.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* srow, int64_t n, uint32_t r, int lane) {
  int64_t lo = 0, len = n;
  while (len > 0) {
    const int64_t step = (len + kWave - 1) / kWave, at = lo + step * lane;
    const int below = __popcll(__ballot(at < lo + len && srow[at < lo + len ? at : lo] < r));   // a prefix of the lanes
    if (below == 0) return lo;
    const int64_t next = lo + step * (below - 1) + 1;
    const int64_t end = lo + step * below;
    len = (end < lo + len ? end : lo + len) - next;
    lo = next;
  }
  return lo;
}

constexpr int kGradRows = 8;   // table rows per wave of the pass over the whole table
constexpr int kGradPos = 4;    // sorted positions per wave of the pass over the named rows

// The whole table: each wave writes kGradRows rows of its columns.
template <bool BF16, bool OUT16, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_table_kernel(const uint32_t* __restrict__ srow,
                                                               const uint32_t* __restrict__ stok, int64_t n_ids,
                                                               const void* dy, const float* part, const float* prev,
                                                               void* packed, uint32_t rows, int64_t cols, float sigma) {
  const int lane = threadIdx.x % kWave;
  const int64_t c0 = (static_cast<int64_t>(blockIdx.y) * (kThreads / kWave) + threadIdx.x / kWave) * kWaveCols;
  if (c0 >= cols) return;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kGradRows;
  int64_t pos = lower_bound(srow, n_ids, static_cast<uint32_t>(r0), lane);
  Window w;
  for (int64_t r = r0; r < r0 + kGradRows && r < rows; ++r) {
    const f32x4 sum = sum_row<BF16, VEC>(static_cast<uint32_t>(r), pos, w, srow, stok, n_ids, dy, part, c0, cols, lane);
    store_row<OUT16, VEC>(packed, prev, r * cols, sum, sigma, c0, cols, lane);
  }
}

// The named rows alone, in place: each wave takes the rows that begin in its
// kGradPos sorted positions.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_named_kernel(const uint32_t* __restrict__ srow,
                                                               const uint32_t* __restrict__ stok, int64_t n_ids,
                                                               const void* dy, const float* part, float* packed,
                                                               int64_t cols, float sigma) {
  const int lane = threadIdx.x % kWave;
  const int64_t c0 = (static_cast<int64_t>(blockIdx.y) * (kThreads / kWave) + threadIdx.x / kWave) * kWaveCols;
  if (c0 >= cols) return;
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kGradPos;
  const int64_t end = p0 + kGradPos < n_ids ? p0 + kGradPos : n_ids;
  Window w;
  int64_t pos = p0;
  uint32_t before = p0 ? srow[p0 - 1] : kNoRow;
  while (pos < end) {
    w.at(pos, srow, stok, n_ids, lane);
    const uint32_t r = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(w.row), static_cast<int>(pos - w.base)));
    if (r == kNoRow) break;              // tokens without a row come last
    if (r == before) {                   // a row that began in front of this wave's positions
      ++pos;
      continue;
    }
    before = r;
    const f32x4 sum = sum_row<BF16, VEC>(r, pos, w, srow, stok, n_ids, dy, part, c0, cols, lane);
    store_row<false, VEC>(packed, packed, static_cast<int64_t>(r) * cols, sum, sigma, c0, cols, lane);
  }
}

// ------------------------------------------------------------------ host

// The table of an embedding call: a tensor of the plan in row-major order.
int check_table(const rs_plan* p, int64_t tensor, int64_t n_ids, const char* who) {
  if (tensor < 0 || tensor >= p->n) return fail(RS_EINVAL, std::string(who) + ": no such tensor");
  const Tensor& t = p->t[tensor];
  if (t.kind == RS_TILEMAJOR) return fail(RS_EINVAL, std::string(who) + ": a TILEMAJOR tensor has no contiguous rows");
  if (n_ids < 0) return fail(RS_EINVAL, std::string(who) + ": negative number of tokens");
  if (t.rows >= (int64_t(1) << 31) || t.cols >= (int64_t(1) << 31) || n_ids >= (int64_t(1) << 31) ||
      n_ids * t.cols > kMaxElems)
    return fail(RS_ERANGE, std::string(who) + ": rows, columns and tokens must be under 2^31, tokens * columns at most 2^39");
  return RS_OK;
}

int check_ids(const void* ids, int32_t id_bytes, int64_t n_ids, const char* who) {
  if (id_bytes != 4 && id_bytes != 8) return fail(RS_EINVAL, std::string(who) + ": token ids have 4 or 8 bytes");
  if (n_ids && !ids) return fail(RS_EINVAL, std::string(who) + ": null token ids");
  if (reinterpret_cast<uintptr_t>(ids) % static_cast<uintptr_t>(id_bytes))
    return fail(RS_EALIGN, std::string(who) + ": token ids must be aligned to their size");
  return RS_OK;
}

struct EmbedWork {
  int64_t keys, srow, stok, part, bytes;
};

EmbedWork embed_work(int64_t n_ids, int64_t cols) {
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  EmbedWork w{};
  w.keys = 0;
  w.srow = w.keys + (n_ids > kRun ? up(8 * n_ids) : 0);
  w.stok = w.srow + up(4 * n_ids);
  w.part = w.stok + up(4 * n_ids);
  w.bytes = w.part + up(n_ids / kSumChunk * cols * 4);
  return w;
}

template <bool IN16, bool OUT16>
void launch_rows(bool vec, const void* table, const void* ids, bool wide, int64_t n_ids, const Tensor& t, float scale,
                 void* out, hipStream_t s) {
  const int64_t units = vec ? t.cols / 8 : t.cols, n = n_ids * units;
  const dim3 grid(static_cast<unsigned>((n + kThreads * kLookVecs - 1) / (kThreads * kLookVecs)));
  if (vec)
    hipLaunchKernelGGL((embed_rows_kernel<IN16, OUT16, true>), grid, dim3(kThreads), 0, s, table, ids, wide, n,
                       static_cast<uint32_t>(units), static_cast<uint32_t>(t.rows), t.cols, scale, out);
  else
    hipLaunchKernelGGL((embed_rows_kernel<IN16, OUT16, false>), grid, dim3(kThreads), 0, s, table, ids, wide, n,
                       static_cast<uint32_t>(units), static_cast<uint32_t>(t.rows), t.cols, scale, out);
}

template <bool BF16, bool VEC>
void launch_grad(const Tensor& t, int64_t n_ids, const void* dy, const float* prev, void* packed, bool out16,
                 float sigma, char* work, hipStream_t s) {
  const EmbedWork w = embed_work(n_ids, t.cols);
  uint32_t* srow = reinterpret_cast<uint32_t*>(work + w.srow);
  uint32_t* stok = reinterpret_cast<uint32_t*>(work + w.stok);
  const int64_t per = kWaveCols * (kThreads / kWave);
  const unsigned pieces = static_cast<unsigned>((t.cols + per - 1) / per);
  float* part = n_ids >= kSumChunk ? reinterpret_cast<float*>(work + w.part) : nullptr;
  if (part)
    hipLaunchKernelGGL((embed_chunk_kernel<BF16, VEC>), dim3(static_cast<unsigned>(n_ids / kSumChunk), pieces),
                       dim3(kThreads), 0, s, srow, stok, n_ids, dy, t.cols, part);
  if (prev == packed) {
    hipLaunchKernelGGL((embed_named_kernel<BF16, VEC>),
                       dim3(static_cast<unsigned>((n_ids + kGradPos - 1) / kGradPos), pieces), dim3(kThreads), 0, s,
                       srow, stok, n_ids, dy, part, static_cast<float*>(packed), t.cols, sigma);
    return;
  }
  const dim3 grid(static_cast<unsigned>((t.rows + kGradRows - 1) / kGradRows), pieces);
  if (out16)
    hipLaunchKernelGGL((embed_table_kernel<BF16, true, VEC>), grid, dim3(kThreads), 0, s, srow, stok, n_ids, dy, part,
                       prev, packed, static_cast<uint32_t>(t.rows), t.cols, sigma);
  else
    hipLaunchKernelGGL((embed_table_kernel<BF16, false, VEC>), grid, dim3(kThreads), 0, s, srow, stok, n_ids, dy, part,
                       prev, packed, static_cast<uint32_t>(t.rows), t.cols, sigma);
}

}  // namespace
}  // namespace rs

using namespace rs;

extern "C" int rs_embed_rows(rs_plan* p, int64_t tensor, const void* gathered, int32_t dt, const void* ids,
                             int32_t id_bytes, int64_t n_ids, float scale, void* out, int32_t out_dt, void* stream) {
  const char* who = "rs_embed_rows";
  clear_error();
  int st = check_call(p, who);
  if (st == RS_OK) st = check_table(p, tensor, n_ids, who);
  if (st == RS_OK) st = check_ids(ids, id_bytes, n_ids, who);
  if (st != RS_OK) return st;
  if (!gathered || (n_ids && !out)) return fail(RS_EINVAL, std::string(who) + ": null argument");
  if ((dt != RS_F32 && dt != RS_BF16) || (out_dt != RS_F32 && out_dt != RS_BF16))
    return fail(RS_EDTYPE, std::string(who) + ": fp32 or bf16");
  if (!std::isfinite(scale)) return fail(RS_EINVAL, std::string(who) + ": scale must be finite");
  if (!aligned16(gathered) || !aligned16(out)) return fail(RS_EALIGN, std::string(who) + ": buffers must be 16-byte aligned");
  if (n_ids == 0) return RS_OK;
  const Tensor& t = p->t[tensor];
  const void* table = static_cast<const char*>(gathered) + t.start * elem_bytes(dt);
  const bool vec = t.cols % 8 == 0, wide = id_bytes == 8;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dt == RS_BF16 && out_dt == RS_BF16) launch_rows<true, true>(vec, table, ids, wide, n_ids, t, scale, out, s);
  else if (dt == RS_BF16) launch_rows<true, false>(vec, table, ids, wide, n_ids, t, scale, out, s);
  else if (out_dt == RS_BF16) launch_rows<false, true>(vec, table, ids, wide, n_ids, t, scale, out, s);
  else launch_rows<false, false>(vec, table, ids, wide, n_ids, t, scale, out, s);
  return launched(who);
}

extern "C" int rs_embed_workspace(const rs_plan* p, int64_t tensor, int64_t n_ids, int64_t* bytes) {
  const char* who = "rs_embed_workspace";
  clear_error();
  if (!p || !bytes) return fail(RS_EINVAL, std::string(who) + ": null argument");
  const int st = check_table(p, tensor, n_ids, who);
  if (st != RS_OK) return st;
  *bytes = embed_work(n_ids, p->t[tensor].cols).bytes;
  return RS_OK;
}

extern "C" int rs_embed_grad(rs_plan* p, int64_t tensor, const void* ids, int32_t id_bytes, int64_t n_ids,
                             const void* dy, int32_t dy_dt, const float* prev, void* packed, int32_t packed_dt,
                             int32_t scale_mode, float scale, void* work, int64_t work_bytes, void* stream) {
  const char* who = "rs_embed_grad";
  clear_error();
  int st = check_call(p, who);
  if (st == RS_OK) st = check_table(p, tensor, n_ids, who);
  if (st == RS_OK) st = check_ids(ids, id_bytes, n_ids, who);
  if (st != RS_OK) return st;
  if ((n_ids && (!dy || !work)) || !packed) return fail(RS_EINVAL, std::string(who) + ": null argument");
  if ((dy_dt != RS_F32 && dy_dt != RS_BF16) || (packed_dt != RS_F32 && packed_dt != RS_BF16))
    return fail(RS_EDTYPE, std::string(who) + ": fp32 or bf16");
  if (prev == packed && packed_dt != RS_F32)
    return fail(RS_EINVAL, std::string(who) + ": prev may be packed only when packed is fp32");
  if ((scale_mode != RS_SCALE_INV_V && scale_mode != RS_SCALE_GIVEN) || !std::isfinite(scale))
    return fail(RS_EINVAL, std::string(who) + ": bad scale");
  if (!aligned16(dy) || !aligned16(prev) || !aligned16(packed) || !aligned16(work))
    return fail(RS_EALIGN, std::string(who) + ": buffers must be 16-byte aligned");
  const Tensor& t = p->t[tensor];
  const EmbedWork w = embed_work(n_ids, t.cols);
  if (work_bytes < w.bytes)
    return fail(RS_EINVAL, std::string(who) + ": workspace of " + std::to_string(work_bytes) + " bytes, " +
                               std::to_string(w.bytes) + " needed");
  if (n_ids == 0 && prev == packed) return RS_OK;
  const float sigma = scale_mode == RS_SCALE_INV_V
                          ? static_cast<float>(static_cast<double>(scale) / static_cast<double>(p->V))
                          : scale;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(work);
  uint32_t* srow = reinterpret_cast<uint32_t*>(ws + w.srow);
  uint32_t* stok = reinterpret_cast<uint32_t*>(ws + w.stok);
  if (n_ids) {
    const int64_t runs = (n_ids + kRun - 1) / kRun;
    int n = 2;
    while (n < std::min<int64_t>(n_ids, kRun)) n *= 2;
    uint64_t* keys = runs > 1 ? reinterpret_cast<uint64_t*>(ws + w.keys) : nullptr;
    hipLaunchKernelGGL(embed_sort_kernel, dim3(static_cast<unsigned>(runs)), dim3(kSortThreads), 0, s, ids,
                       id_bytes == 8, n_ids, static_cast<uint32_t>(t.rows), n, keys, srow, stok);
    if (runs > 1)
      hipLaunchKernelGGL(embed_merge_kernel, dim3(static_cast<unsigned>((n_ids + kThreads - 1) / kThreads)),
                         dim3(kThreads), 0, s, keys, n_ids, srow, stok);
  }
  void* out = static_cast<char*>(packed) + t.start * elem_bytes(packed_dt);
  const float* pv = prev ? prev + t.start : nullptr;
  const bool vec = t.cols % 4 == 0, out16 = packed_dt == RS_BF16;
  if (dy_dt == RS_BF16 && vec) launch_grad<true, true>(t, n_ids, dy, pv, out, out16, sigma, ws, s);
  else if (dy_dt == RS_BF16) launch_grad<true, false>(t, n_ids, dy, pv, out, out16, sigma, ws, s);
  else if (vec) launch_grad<false, true>(t, n_ids, dy, pv, out, out16, sigma, ws, s);
  else launch_grad<false, false>(t, n_ids, dy, pv, out, out16, sigma, ws, s);
  return launched(who);
}
