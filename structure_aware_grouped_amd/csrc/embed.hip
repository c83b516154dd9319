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
// the tokens are sorted by row, in their own order within a row; whole chunks
// of 64 sorted tokens of one row (common tokens) are summed by workgroups of
// their own; then each row adds its chunk sums and its remaining tokens in
// order.
#include "host_common.h"

#include <algorithm>
#include <type_traits>

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

// Bound by memory: 16384 tokens of 8192 bf16 columns take 91 us, 5.9 TB/s with
// every token's row counted, as a copy does, whatever the vectors a thread
// (2, 4 and 8 alike, one 104 us), the cache policy or the XCD order. Of the 255
// MB of rows that its tokens name, 109 MB of them different, 193 MB come from
// HBM: other XCDs read a repeated row again.
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

// ------------------------------------------------------------------ fill

// Elements [from, to) of the tensor's interval <- prev + 0.0, or +0.0. Where
// few rows are named, this and a pass over the named rows are faster than one
// pass that looks for tokens of every row (131072 x 4096, 16384 tokens: 370 us
// instead of 554). The fill runs as the tail of the grids of the sort and of
// the chunk sums, which are short of workgroups and wait for memory (the
// merge's 64 KiB of LDS would leave room for few fill blocks). The sort takes
// kSortFill bytes of it or a sixteenth, about what is moved while the runs are
// sorted: a 32001 x 1001 bf16 table with 4097 tokens took 43 us with the
// sixteenth and 38.5 with 64 or 96 MiB; 131072 x 4096 took 375 us with 32 MiB,
// 371 with 64, 368 with 96 and 369 with the sixteenth (128). One 16-byte
// nt-sc1 store a thread in workgroups of 256 filled 2 GiB at 7.16 TB/s, four a
// thread at 6.07, 64 threads at 4.82.
constexpr int64_t kSortFill = int64_t(96) << 20;
struct Fill {
  const float* prev;
  void* packed;
  int64_t from, to;   // from: a multiple of 16
  bool out16;
};

// elements of one block
constexpr int64_t fill_piece(int threads, bool out16) { return int64_t(threads) * (out16 ? 8 : 4); }

template <int NT>
__device__ __forceinline__ void fill_block(const Fill& f, int64_t block) {
  const int64_t first = f.from + block * fill_piece(NT, f.out16);
  if (f.out16) {
    const int64_t e = first + threadIdx.x * 8;
    float v[8] = {};
    if (e + 8 <= f.to) {
      if (f.prev) {
        load8<false>(f.prev, e, v);
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = __fadd_rn(v[t], 0.0f);
      }
      uint32_t b[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) b[t] = bf16_rne(v[t]);
      sts_at<kStoreNtSc1>(static_cast<uint16_t*>(f.packed) + first, threadIdx.x * 16,
                          u32x4{b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16});
    } else {
      for (int64_t t = e; t < f.to; ++t)
        static_cast<uint16_t*>(f.packed)[t] = static_cast<uint16_t>(bf16_rne(f.prev ? __fadd_rn(f.prev[t], 0.0f) : 0.0f));
    }
  } else {
    const int64_t e = first + threadIdx.x * 4;
    f32x4 v = {};
    if (e + 4 <= f.to) {
      if (f.prev) {
        v = ldg(reinterpret_cast<const f32x4*>(f.prev + e));
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = __fadd_rn(v[t], 0.0f);
      }
      sts_at<kStoreNtSc1>(static_cast<float*>(f.packed) + first, threadIdx.x * 16, v);
    } else {
      for (int64_t t = e; t < f.to; ++t) static_cast<float*>(f.packed)[t] = f.prev ? __fadd_rn(f.prev[t], 0.0f) : 0.0f;
    }
  }
}

// ------------------------------------------------------------------ sort

constexpr int kRun = 2048;            // tokens sorted in LDS by one workgroup
constexpr int kSortThreads = 1024;
constexpr int kSortGroups = kRun / kWave;
constexpr int kDigitBits = 6, kDigits = 1 << kDigitBits;
constexpr int kSumChunk = 64;         // sorted tokens of one row summed ahead
static_assert(kDigits * kSortGroups == 2 * kSortThreads && kRun == 2 * kSortThreads, "two counters and tokens a thread");

// kRun tokens sorted by row in LDS, in their own order within a row: a radix
// sort from the lowest six bits up, `passes` times. A group of 64 neighbours
// finds equal digits by ballots; the counters, by digit and then group, are
// added up in front of each other, and a token's place is its counter's sum
// plus its rank among the group's equals. A bitonic network of the same 2048
// took 21 us, most of it barriers.
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(const void* ids, bool wide, int64_t n_ids,
                                                                  uint32_t rows, int passes, uint32_t* out_row,
                                                                  uint32_t* out_tok, unsigned runs, Fill fill) {
  __shared__ uint32_t key[2][kRun];
  __shared__ uint16_t idx[2][kRun];
  __shared__ uint32_t count[kDigits * kSortGroups];
  __shared__ uint32_t wave_sum[kSortThreads / kWave];
  if (blockIdx.x >= runs) {
    fill_block<kSortThreads>(fill, blockIdx.x - runs);
    return;
  }
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kRun;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = (wave * 2 + k) * kWave + lane;
    key[0][i] = base + i < n_ids ? row_of(ids, wide, base + i, rows) : kNoRow;
    idx[0][i] = static_cast<uint16_t>(i);
  }
  int from = 0;
  for (int p = 0; p < passes; ++p) {
    for (int i = tid; i < kDigits * kSortGroups; i += kSortThreads) count[i] = 0;
    __syncthreads();
    uint32_t row[2], tok[2], rank[2], slot[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int group = wave * 2 + k, i = group * kWave + lane;
      row[k] = key[from][i];
      tok[k] = idx[from][i];
      const uint32_t digit = row[k] >> (p * kDigitBits) & (kDigits - 1);
      uint64_t equal = ~0ull;
#pragma unroll
      for (int b = 0; b < kDigitBits; ++b) {
        const uint64_t set = __ballot(digit >> b & 1);
        equal &= digit >> b & 1 ? set : ~set;
      }
      rank[k] = __popcll(equal & ((1ull << lane) - 1));
      slot[k] = digit * kSortGroups + group;
      if (rank[k] == 0) count[slot[k]] = __popcll(equal);
    }
    __syncthreads();
    // exclusive sums over the counters, two neighbours a thread
    const uint32_t c0 = count[2 * tid], c1 = count[2 * tid + 1];
    uint32_t sum = c0 + c1;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const uint32_t up = __shfl_up(sum, o, kWave);
      if (lane >= o) sum += up;
    }
    if (lane == kWave - 1) wave_sum[wave] = sum;
    __syncthreads();
    uint32_t waves = lane < wave ? wave_sum[lane] : 0u;   // of the waves in front, 15 at most
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) waves += __shfl_xor(waves, o, kWave);
    const uint32_t before = sum - c0 - c1 + __shfl(waves, 0, kWave);
    count[2 * tid] = before;
    count[2 * tid + 1] = before + c0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t to = count[slot[k]] + rank[k];
      key[from ^ 1][to] = row[k];
      idx[from ^ 1][to] = static_cast<uint16_t>(tok[k]);
    }
    from ^= 1;
    __syncthreads();
  }
  // what lies behind the last token sorted behind the ids that name no row,
  // which it equals: those come first, in their own order
  for (int i = tid; i < kRun && base + i < n_ids; i += kSortThreads) {
    out_row[base + i] = key[from][i];
    out_tok[base + i] = static_cast<uint32_t>(base) + idx[from][i];
  }
}

// Sorted runs -> one sorted list of each `span` neighbouring runs: a token's
// place is its place in its own run plus, in every other run, the number of
// smaller rows, or of smaller and equal rows where that run's tokens come
// first. The runs' rows are searched in LDS, kMergeRuns at a time (in memory
// the 11 dependent reads of one search took 15 us).
constexpr int kMergeRuns = 8;
constexpr int64_t kMergeAll = 16;   // runs merged in one launch (32: 94 us so, 80 in two passes; 16: 60 either way)

__global__ __launch_bounds__(kThreads) void embed_merge_kernel(const uint32_t* __restrict__ rows,
                                                               const uint32_t* __restrict__ toks, int64_t n_ids,
                                                               int64_t span, uint32_t* srow, uint32_t* stok) {
  __shared__ __attribute__((aligned(16))) uint32_t s[kMergeRuns][kRun];
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const bool in = i < n_ids;
  const uint32_t row = in ? rows[i] : 0u, tok = in ? toks[i] : 0u;
  const int64_t own = i / kRun, begin = own / span * span, end = begin + span;
  int64_t place = i - own * kRun + begin * kRun;
  for (int64_t r0 = begin; r0 < end && r0 * kRun < n_ids; r0 += kMergeRuns) {
    __syncthreads();
    uint32_t* flat = &s[0][0];
    const int64_t at = r0 * kRun;
    const int here = static_cast<int>(n_ids - at < kMergeRuns * kRun ? n_ids - at : kMergeRuns * kRun);
#pragma unroll 8
    for (int e = threadIdx.x * 4; e < here / 4 * 4; e += kThreads * 4)
      *reinterpret_cast<u32x4*>(flat + e) = *reinterpret_cast<const u32x4*>(rows + at + e);
    if (static_cast<int>(threadIdx.x) < here % 4) flat[here / 4 * 4 + threadIdx.x] = rows[at + here / 4 * 4 + threadIdx.x];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kMergeRuns; ++r) {
      // rows below `row` (or not above it) lie in front of lo
      const int64_t first = at + r * kRun;
      const int len = first >= n_ids || r0 + r == own ? 0 : static_cast<int>(n_ids - first < kRun ? n_ids - first : kRun);
      const bool equal = r0 + r < own;
      int lo = 0;
#pragma unroll
      for (int step = kRun; step > 0; step /= 2) {
        const int next = lo + step;
        if (next <= len) {
          const uint32_t x = s[r][next - 1];
          if (equal ? x <= row : x < row) lo = next;
        }
      }
      place += lo;
    }
  }
  if (in) {
    srow[place] = row;
    stok[place] = tok;
  }
}

// One more pass over sorted lists of len = kRun * kMergeRuns^k tokens: each
// kMergeRuns neighbouring ones -> one, as above, with the searches in memory.
// A thread's searches in the other lists go step by step together, and a
// wave's tokens, neighbours in a sorted list, read neighbouring places.
__global__ __launch_bounds__(kThreads) void embed_merge_lists_kernel(const uint32_t* __restrict__ rows,
                                                                     const uint32_t* __restrict__ toks, int n_ids,
                                                                     int len, uint32_t* srow, uint32_t* stok) {
  const int i = static_cast<int>(blockIdx.x) * kThreads + static_cast<int>(threadIdx.x);
  if (i >= n_ids) return;
  const uint32_t row = rows[i];
  const int own = i / len, begin = own / kMergeRuns * kMergeRuns;
  int lo[kMergeRuns], size[kMergeRuns];
#pragma unroll
  for (int r = 0; r < kMergeRuns; ++r) {
    const int64_t first = static_cast<int64_t>(begin + r) * len;
    lo[r] = 0;
    size[r] = first >= n_ids || begin + r == own ? 0 : static_cast<int>(n_ids - first < len ? n_ids - first : len);
  }
  for (int step = len; step > 0; step /= 2) {
#pragma unroll
    for (int r = 0; r < kMergeRuns; ++r) {
      const int next = lo[r] + step;
      if (next <= size[r]) {
        const uint32_t x = rows[static_cast<int64_t>(begin + r) * len + next - 1];
        if (begin + r < own ? x <= row : x < row) lo[r] = next;
      }
    }
  }
  int place = i - own * len + begin * len;
#pragma unroll
  for (int r = 0; r < kMergeRuns; ++r) place += lo[r];
  srow[place] = row;
  stok[place] = toks[i];
}

// ------------------------------------------------------------------ gradient

// Columns of one wave: lane l holds four. Whole vectors of four neighbours
// where the width is a multiple of 4, else single columns 64 apart.
constexpr int kWaveCols = 4 * kWave;

template <bool VEC>
__device__ __forceinline__ int64_t col_of(int64_t c0, int lane, int e) {
  return VEC ? c0 + lane * 4 + e : c0 + e * kWave + lane;
}

// Lanes past the width read its last columns, which they do not store: a
// branch around every load would keep the loads from going out together.
template <bool BF16, bool VEC>
__device__ __forceinline__ f32x4 load_cols(const void* p, int64_t row_at, int64_t c0, int64_t cols, int lane) {
  f32x4 x;
  if constexpr (VEC) {
    const int64_t at = row_at + min(c0 + lane * 4, cols - 4);
    if constexpr (BF16) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + at);
      x = f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                __uint_as_float(w.y & 0xffff0000u)};
    } else {
      x = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = In<BF16>::elem(p, row_at + min(col_of<false>(c0, lane, e), cols - 1));
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
  auto add = [&](auto count) {
    constexpr int N = decltype(count)::value;
    for (; i + N <= to; i += N) {
      f32x4 x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const uint32_t t = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(w.tok), i + k));
        x[k] = load_cols<BF16, VEC>(dy, static_cast<int64_t>(t) * cols, c0, cols, lane);
      }
#pragma unroll
      for (int k = 0; k < N; ++k) sum += x[k];
    }
  };
  add(std::integral_constant<int, 16>{});   // rows on their way at a time
  add(std::integral_constant<int, 4>{});
  add(std::integral_constant<int, 1>{});
  return sum;
}

// Chunks of kSumChunk sorted tokens that are all one row's -> their sums.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_chunk_kernel(const uint32_t* __restrict__ srow,
                                                               const uint32_t* __restrict__ stok, int64_t n_ids,
                                                               const void* dy, int64_t cols, float* part,
                                                               unsigned chunks, unsigned pieces, Fill fill) {
  if (blockIdx.x >= chunks * pieces) {
    fill_block<kThreads>(fill, blockIdx.x - chunks * pieces);
    return;
  }
  const int lane = threadIdx.x % kWave;
  const int64_t chunk = blockIdx.x / pieces;
  Window w;
  w.at(chunk * kSumChunk, srow, stok, n_ids, lane);
  const uint32_t first = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(w.row)));
  if (first == kNoRow || !__all(w.row == first)) return;
  const int64_t c0 = (static_cast<int64_t>(blockIdx.x % pieces) * (kThreads / kWave) + threadIdx.x / kWave) * kWaveCols;
  if (c0 >= cols) return;
  const f32x4 sum = sum_tokens<BF16, VEC>(f32x4{}, w, 0, kSumChunk, dy, c0, cols, lane);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t c = col_of<VEC>(c0, lane, e);
    if (c < cols) part[chunk * cols + c] = sum[e];
  }
}

// Sum over the tokens of row r from sorted position pos on; moves pos past them.
// A wave goes through the row's 64-token windows one by one, each a dependent
// load of the window and one of its chunk sum, so a row that very many tokens
// name takes 0.5 to 0.6 us for every 64 of them: 65536 tokens of one row 506 us
// the call (spread by a power law 80), 2^20 of them 10 ms (0.9).
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
    if (part && count == kSumChunk) {
      sum += load_cols<false, VEC>(part, w.base / kSumChunk * cols, c0, cols, lane);
    } else
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
constexpr int kGradPos = 8;    // sorted positions per wave of the pass over the named rows
// The whole table: each wave writes kGradRows rows of its columns.
template <bool BF16, bool OUT16, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_table_kernel(const uint32_t* __restrict__ srow,
                                                               const uint32_t* __restrict__ stok, int64_t n_ids,
                                                               const void* dy, const float* part, const float* prev,
                                                               void* packed, uint32_t rows, int64_t cols, float sigma,
                                                               unsigned pieces) {
  const int lane = threadIdx.x % kWave;
  const int64_t c0 = (static_cast<int64_t>(blockIdx.x % pieces) * (kThreads / kWave) + threadIdx.x / kWave) * kWaveCols;
  if (c0 >= cols) return;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x / pieces) * kGradRows;
  int64_t pos = lower_bound(srow, n_ids, static_cast<uint32_t>(r0), lane);
  Window w;
  for (int64_t r = r0; r < r0 + kGradRows && r < rows; ++r) {
    const int64_t first = pos;
    const f32x4 sum = sum_row<BF16, VEC>(static_cast<uint32_t>(r), pos, w, srow, stok, n_ids, dy, part, c0, cols, lane);
    // a row that no token names gets +0.0 or prev + 0.0, as from the fill: a negative sigma would make it -0.0
    store_row<OUT16, VEC>(packed, prev, r * cols, sum, pos == first ? 0.0f : sigma, c0, cols, lane);
  }
}

// The named rows alone: each wave takes the rows that begin in its kGradPos
// sorted positions. The tokens of all its positions are on their way together;
// a row that goes on behind them is summed by itself.
template <bool BF16, bool OUT16, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_named_kernel(const uint32_t* __restrict__ srow,
                                                               const uint32_t* __restrict__ stok, int64_t n_ids,
                                                               const void* dy, const float* part, const float* prev,
                                                               void* packed, int64_t cols, float sigma,
                                                               unsigned pieces) {
  static_assert(kSumChunk % kGradPos == 0, "a wave's positions lie in one window");
  const int lane = threadIdx.x % kWave;
  const int64_t c0 = (static_cast<int64_t>(blockIdx.x % pieces) * (kThreads / kWave) + threadIdx.x / kWave) * kWaveCols;
  if (c0 >= cols) return;
  const int64_t p0 = static_cast<int64_t>(blockIdx.x / pieces) * kGradPos;
  Window w;
  w.at(p0, srow, stok, n_ids, lane);
  const uint32_t before = p0 ? srow[p0 - 1] : kNoRow, behind = p0 + kGradPos < n_ids ? srow[p0 + kGradPos] : kNoRow;
  const int at = static_cast<int>(p0 - w.base);
  uint32_t row[kGradPos + 1];
  f32x4 x[kGradPos];
#pragma unroll
  for (int k = 0; k < kGradPos; ++k) {
    row[k] = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(w.row), at + k));   // kNoRow behind the last token
    const uint32_t t = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(w.tok), at + k));
    x[k] = f32x4{};
    if (row[k] != kNoRow && row[k] != before) x[k] = load_cols<BF16, VEC>(dy, static_cast<int64_t>(t) * cols, c0, cols, lane);
  }
  row[kGradPos] = behind;
  f32x4 sum = {};
  int start = 0;
#pragma unroll
  for (int k = 0; k < kGradPos; ++k) {
    if (row[k] == kNoRow || row[k] == before) continue;   // no row, or one that began in front of these positions
    if (k == 0 || row[k] != row[k - 1]) {
      sum = f32x4{};
      start = k;
    }
    sum += x[k];
    if (row[k] == row[k + 1]) {
      if (k + 1 < kGradPos) continue;
      int64_t pos = p0 + start;
      sum = sum_row<BF16, VEC>(row[k], pos, w, srow, stok, n_ids, dy, part, c0, cols, lane);
    }
    store_row<OUT16, VEC>(packed, prev, static_cast<int64_t>(row[k]) * cols, sum, sigma, c0, cols, lane);
  }
}

// ------------------------------------------------------------------ host

// Limits that keep every launch under 2^32 work-items: 32 per row (whole
// groups of kGradRows) or token in the gradient's passes, a quarter per element
// in the fill and the lookup. The lookup numbers a row's units in 32 bits.
constexpr int64_t kEmbedMaxRows = (int64_t(1) << 27) - kGradRows, kEmbedMaxCols = int64_t(1) << 31;
constexpr int64_t kEmbedMaxIds = int64_t(1) << 26;
static_assert((kEmbedMaxRows + kGradRows - 1) / kGradRows * kThreads < int64_t(1) << 32, "the whole-table pass");
constexpr int64_t kEmbedMaxTable = int64_t(1) << 34, kEmbedMaxElems = int64_t(1) << 33;

// The table of an embedding call: a tensor of the plan in row-major order.
int check_table(const rs_plan* p, int64_t tensor, int64_t n_ids, const char* who) {
  if (tensor < 0 || tensor >= p->n) return fail(RS_EINVAL, std::string(who) + ": no such tensor");
  const Tensor& t = p->t[tensor];
  if (t.kind == RS_TILEMAJOR) return fail(RS_EINVAL, std::string(who) + ": a TILEMAJOR tensor has no contiguous rows");
  if (n_ids < 0) return fail(RS_EINVAL, std::string(who) + ": negative number of tokens");
  if (t.rows > kEmbedMaxRows || t.cols >= kEmbedMaxCols || t.n > kEmbedMaxTable || n_ids >= kEmbedMaxIds ||
      n_ids * t.cols > kEmbedMaxElems)
    return fail(RS_ERANGE, std::string(who) + ": rows at most 2^27 - 8, columns under 2^31, table at most 2^34 "
                               "elements, tokens under 2^26, tokens * columns at most 2^33");
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
  int64_t rrow, rtok, srow, stok, part, bytes;   // sorted runs, sorted list, chunk sums
};

EmbedWork embed_work(int64_t n_ids, int64_t cols) {
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  EmbedWork w{};
  const int64_t list = up(4 * n_ids), runs = n_ids > kRun ? list : 0;
  w.rrow = 0;
  w.rtok = w.rrow + runs;
  w.srow = w.rtok + runs;
  w.stok = w.srow + list;
  w.part = w.stok + list;
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

struct GradCall {
  const void* ids;
  bool wide;
  int64_t n_ids;
  const void* dy;
  const float* prev;   // of the tensor's interval, like packed
  void* packed;
  bool out16;
  float sigma;
  char* work;
};

template <bool BF16, bool VEC>
void launch_grad(const Tensor& t, const GradCall& c, hipStream_t s) {
  const int64_t n = c.n_ids;
  const EmbedWork w = embed_work(n, t.cols);
  uint32_t* srow = reinterpret_cast<uint32_t*>(c.work + w.srow);
  uint32_t* stok = reinterpret_cast<uint32_t*>(c.work + w.stok);
  const int64_t per = kWaveCols * (kThreads / kWave);
  const unsigned pieces = static_cast<unsigned>((t.cols + per - 1) / per);
  const int64_t runs = (n + kRun - 1) / kRun;
  float* part = n >= kSumChunk ? reinterpret_cast<float*>(c.work + w.part) : nullptr;
  const bool in_place = c.prev == c.packed, named = in_place || n < t.rows / 2;
  // the fill, in shares of the launches ahead of the named rows' pass; the
  // chunk sums' launch takes the rest, with or without chunks
  const int64_t fill = named && !in_place ? t.n : 0;
  int64_t filled = 0;
  auto share = [&](int64_t to, int threads, unsigned* blocks) {
    const Fill f = {c.prev, c.packed, filled, to, c.out16};
    *blocks = static_cast<unsigned>((to - filled + fill_piece(threads, c.out16) - 1) / fill_piece(threads, c.out16));
    filled = to;
    return f;
  };
  unsigned extra = 0;
  // at least a sixteenth: the chunk sums' launch then stays under 2^32 work-items
  const int64_t early = std::max(kSortFill / ((c.out16 ? 2 : 4) + (c.prev ? 4 : 0)), fill / 16 / 16 * 16);
  Fill f = share(std::min(fill, early), kSortThreads, &extra);
  // digits that tell the rows apart from each other and from kNoRow, whose low
  // digits are all ones
  int passes = 1;
  while (passes * kDigitBits < 32 && t.rows >> (passes * kDigitBits) > 0) ++passes;
  // Up to kMergeAll runs are merged at once, which reads all of them for every
  // 256 tokens; more in passes of kMergeRuns, so that the time stays in
  // proportion to the tokens (131072 of them at once 177 us the call, in passes
  // 133; 2^20 5.5 ms and 0.91). The passes go to and fro between two lists and
  // end in srow.
  int merges = runs > 1 ? 1 : 0;
  if (runs > kMergeAll)
    for (int64_t lists = (runs + kMergeRuns - 1) / kMergeRuns; lists > 1; lists = (lists + kMergeRuns - 1) / kMergeRuns) ++merges;
  uint32_t* list_row[2] = {srow, reinterpret_cast<uint32_t*>(c.work + w.rrow)};
  uint32_t* list_tok[2] = {stok, reinterpret_cast<uint32_t*>(c.work + w.rtok)};
  int from = merges % 2;
  if (runs + extra)
    hipLaunchKernelGGL(embed_sort_kernel, dim3(static_cast<unsigned>(runs) + extra), dim3(kSortThreads), 0, s, c.ids,
                       c.wide, n, static_cast<uint32_t>(t.rows), passes, list_row[from], list_tok[from],
                       static_cast<unsigned>(runs), f);
  const dim3 merge_grid(static_cast<unsigned>((n + kThreads - 1) / kThreads));
  for (int64_t m = 0, len = kRun; m < merges; ++m, len *= kMergeRuns, from ^= 1) {
    if (m == 0)
      hipLaunchKernelGGL(embed_merge_kernel, merge_grid, dim3(kThreads), 0, s, list_row[from], list_tok[from], n,
                         merges == 1 ? runs : int64_t(kMergeRuns), list_row[from ^ 1], list_tok[from ^ 1]);
    else
      hipLaunchKernelGGL(embed_merge_lists_kernel, merge_grid, dim3(kThreads), 0, s, list_row[from], list_tok[from],
                         static_cast<int>(n), static_cast<int>(len), list_row[from ^ 1], list_tok[from ^ 1]);
  }
  const unsigned chunks = static_cast<unsigned>(n / kSumChunk);
  f = share(fill, kThreads, &extra);
  if (chunks + extra)
    hipLaunchKernelGGL((embed_chunk_kernel<BF16, VEC>), dim3(chunks * pieces + extra), dim3(kThreads), 0, s, srow, stok,
                       n, c.dy, t.cols, part, chunks, pieces, f);
  if (named) {
    if (n == 0) return;
    const dim3 grid(static_cast<unsigned>((n + kGradPos - 1) / kGradPos) * pieces);
    if (c.out16)
      hipLaunchKernelGGL((embed_named_kernel<BF16, true, VEC>), grid, dim3(kThreads), 0, s, srow, stok, n, c.dy, part,
                         c.prev, c.packed, t.cols, c.sigma, pieces);
    else
      hipLaunchKernelGGL((embed_named_kernel<BF16, false, VEC>), grid, dim3(kThreads), 0, s, srow, stok, n, c.dy, part,
                         c.prev, c.packed, t.cols, c.sigma, pieces);
    return;
  }
  const dim3 grid(static_cast<unsigned>((t.rows + kGradRows - 1) / kGradRows) * pieces);
  if (c.out16)
    hipLaunchKernelGGL((embed_table_kernel<BF16, true, VEC>), grid, dim3(kThreads), 0, s, srow, stok, n, c.dy, part,
                       c.prev, c.packed, static_cast<uint32_t>(t.rows), t.cols, c.sigma, pieces);
  else
    hipLaunchKernelGGL((embed_table_kernel<BF16, false, VEC>), grid, dim3(kThreads), 0, s, srow, stok, n, c.dy, part,
                       c.prev, c.packed, static_cast<uint32_t>(t.rows), t.cols, c.sigma, pieces);
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
  void* out = static_cast<char*>(packed) + t.start * elem_bytes(packed_dt);
  const GradCall c = {ids, id_bytes == 8, n_ids, dy, prev ? prev + t.start : nullptr, out, packed_dt == RS_BF16, sigma,
                      static_cast<char*>(work)};
  const bool vec = t.cols % 4 == 0;
  if (dy_dt == RS_BF16 && vec) launch_grad<true, true>(t, c, s);
  else if (dy_dt == RS_BF16) launch_grad<true, false>(t, c, s);
  else if (vec) launch_grad<false, true>(t, c, s);
  else launch_grad<false, false>(t, c, s);
  return launched(who);
}
