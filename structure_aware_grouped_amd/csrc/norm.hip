// Layer norm with its weight and bias read from the gathered flat buffer, and
// its backward pass with their gradients summed into the packed flat buffer,
// on gfx950: kernels and the rs_layer_norm / rs_layer_norm_grad /
// rs_layer_norm_workspace entry points. The weight is used where the gather
// left it and its gradient lands where the reduction reads it
// ("veScale-FSDP: flexible, structure-aware sharding at 10K-GPU scale",
// feynmanwiki walkthrough, DBuffer paragraphs: a tensor is its planned slice).
//
// Mathematics, for a row x of C columns (m = 0 where it is not centred):
//   m = sum x / C,  r = 1 / sqrt(sum (x - m)^2 / C + eps),  h = (x - m) r
//   y = h w + b
// backwards, with g = dy w:
//   dx = r (g - sum(g) / C - h sum(g h) / C)      (no sum(g) where not centred)
//   dw = sum over rows of dy h,   db = sum over rows of dy
//
// Both move bytes only. A workgroup holds a row in registers, so it is read
// once whatever the sums need: the variance is that of the deviations, not a
// difference of squares. The backward pass computes m and r again from the row
// it needs anyway; nothing is kept from the forward pass. A workgroup takes
// every G-th row and adds up its rows' share of dw and db in registers (fp32);
// a second launch adds the G shares in their order, without atomics.
#include "host_common.h"
#include "mfma.h"

namespace rs {
namespace {

// 8 * VPT values of a row per thread, as loaded. VEC: vectors of 8 neighbours
// (every row 16-byte aligned), vector k of thread t is number k * NT + t;
// else value 8 * k + e of thread t is column (8 * k + e) * NT + t.
template <bool STREAM>
__device__ __forceinline__ u32x4 load16(const u32x4* p) {
  if constexpr (STREAM) return ldg(p);
  else return *p;
}

template <bool B16, bool VEC, int VPT, bool STREAM = false>
struct Row {
  u32x4 v[VPT][B16 && VEC ? 1 : 2];

  __device__ __forceinline__ void load(const void* p, int64_t at, int cols, int nt) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if constexpr (VEC) {
        const int c = (k * nt + static_cast<int>(threadIdx.x)) * 8;
        if (c < cols) {
          if constexpr (B16) {
            v[k][0] = load16<STREAM>(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at + c));
          } else {
            const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + at + c);
            v[k][0] = load16<STREAM>(q);
            v[k][1] = load16<STREAM>(q + 1);
          }
        } else {
          v[k][0] = u32x4{};
          if constexpr (!B16) v[k][1] = u32x4{};
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = (k * 8 + e) * nt + static_cast<int>(threadIdx.x);
          v[k][e / 4][e % 4] = c < cols ? __float_as_uint(In<B16>::elem(p, at + c)) : 0u;
        }
      }
    }
  }
  // Keeps the compiler from keeping the widened values across a loop.
  __device__ __forceinline__ void hide() {
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (u32x4& x : v[k]) asm volatile("" : "+v"(x));
  }
  __device__ __forceinline__ void widen(int k, float (&x)[8]) const {
    if constexpr (B16 && VEC) {
      In<true>::widen(v[k][0], x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(v[k][e / 4][e % 4]);
    }
  }
};

// Whether value e of vector k of this thread lies in the row.
template <bool VEC>
__device__ __forceinline__ bool in_row(int k, int e, int cols, int nt) {
  return VEC ? (k * nt + static_cast<int>(threadIdx.x)) * 8 < cols : (k * 8 + e) * nt + static_cast<int>(threadIdx.x) < cols;
}

template <bool B16, bool VEC, int POLICY = 0>
__device__ __forceinline__ void store8(void* p, int64_t at, int k, const float (&x)[8], int cols, int nt) {
  if constexpr (VEC) {
    const int c = (k * nt + static_cast<int>(threadIdx.x)) * 8;
    if (c >= cols) return;
    if constexpr (B16) {
      sts_at<POLICY>(static_cast<uint16_t*>(p) + at, c * 2, u32x4{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7])});
    } else {
      sts_at<POLICY>(static_cast<float*>(p) + at, c * 4, f32x4{x[0], x[1], x[2], x[3]});
      sts_at<POLICY>(static_cast<float*>(p) + at, c * 4 + 16, f32x4{x[4], x[5], x[6], x[7]});
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = (k * 8 + e) * nt + static_cast<int>(threadIdx.x);
      if (c >= cols) continue;
      if constexpr (B16) static_cast<uint16_t*>(p)[at + c] = static_cast<uint16_t>(bf16_rne(x[e]));
      else static_cast<float*>(p)[at + c] = x[e];
    }
  }
}

// Sums over the workgroup, N of them at once, the same bits in every thread.
// `red` alternates between two halves from call to call: whoever writes one
// half has passed the barrier behind the reads of it.
constexpr int kNormThreads = 512, kGradThreads = 1024, kMaxWaves = 16;
static_assert(kGradThreads <= kMaxWaves * kWave, "a row of lanes holds one value of each wave");
template <int N>
__device__ __forceinline__ void group_sum(float (&s)[N], float* red, int& half, int nt) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = wave_sum(s[i]);
  if (nt == kWave) return;
  float* mine = red + half * (2 * kMaxWaves);
  half ^= 1;
  const int lane = static_cast<int>(threadIdx.x) % kWave, wave = static_cast<int>(threadIdx.x) / kWave;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) mine[i * kMaxWaves + wave] = s[i];
  wait<63, true>();
  barrier();
  const int slot = lane % kMaxWaves;
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = from_lane(row_sum_last(slot < nt / kWave ? mine[i * kMaxWaves + slot] : 0.0f), kMaxWaves - 1);
}

// One of the parameters, the same columns as a Row's; zeros where there is none.
template <bool VEC, int VPT>
__device__ __forceinline__ void load_param(const void* p, bool b16, float (&w)[VPT][8], int cols, int nt) {
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    if (p && b16) {
      Row<true, VEC, 1> r;
      r.load(p, static_cast<int64_t>(k) * 8 * nt, cols - k * 8 * nt, nt);
      r.widen(0, w[k]);
    } else if (p) {
      Row<false, VEC, 1> r;
      r.load(p, static_cast<int64_t>(k) * 8 * nt, cols - k * 8 * nt, nt);
      r.widen(0, w[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[k][e] = 0.0f;
    }
  }
}

// Deviations from the mean and the reciprocal deviation of the row.
template <bool B16, bool VEC, int VPT, bool STREAM>
__device__ __forceinline__ float standardize(const Row<B16, VEC, VPT, STREAM>& row, float (&h)[VPT][8], int cols, float eps, bool center,
                                             float* red, int& half, int nt) {
  float s[1] = {0.0f};
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    row.widen(k, h[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] += h[k][e];   // 0 outside the row
  }
  const float width = static_cast<float>(cols);
  if (center) {
    group_sum<1>(s, red, half, nt);
    const float m = s[0] / width;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = in_row<VEC>(k, e, cols, nt) ? h[k][e] - m : 0.0f;
  }
  s[0] = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] = __builtin_fmaf(h[k][e], h[k][e], s[0]);
  group_sum<1>(s, red, half, nt);
  const float r = 1.0f / __builtin_sqrtf(s[0] / width + eps);
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) h[k][e] *= r;
  return r;
}

struct NormCall {
  const void *weight, *bias;   // bias may be null
  bool param16;
  int64_t n;
  int cols;
  float eps;
  bool center;
};

// y of every G-th row. Bound by memory: 16384 rows of 8192 bf16 in 80 to 82 us, 6.6
// TB/s (a call 94), with streaming stores that no barrier waits for. Widths that are
// no multiple of 8 by their single-element accesses: 4097 bf16 rows of 1001, 5001 and
// 9001 in 17, 118 and 210 us a call; above 8192 these spill 14 registers.
template <bool IN16, bool OUT16, bool VEC, int VPT>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(NormCall c, const void* x, void* y) {
  __shared__ __attribute__((aligned(16))) float red[4 * kMaxWaves];
  const int nt = static_cast<int>(blockDim.x);
  int half = 0;
  float w[VPT][8], b[VPT][8];
  load_param<VEC, VPT>(c.weight, c.param16, w, c.cols, nt);
  load_param<VEC, VPT>(c.bias, c.param16, b, c.cols, nt);
  Row<IN16, VEC, VPT> row;
  row.load(x, blockIdx.x * static_cast<int64_t>(c.cols), c.cols, nt);
  for (int64_t r = blockIdx.x; r < c.n; r += gridDim.x) {
    float h[VPT][8];
    standardize(row, h, c.cols, c.eps, c.center, red, half, nt);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (c.bias) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[k][e] = h[k][e] * w[k][e] + b[k][e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[k][e] *= w[k][e];
      }
      store8<OUT16, VEC, kStoreNtSc1>(y, r * c.cols, k, h[k], c.cols, nt);
    }
    if (r + gridDim.x < c.n) row.load(x, (r + gridDim.x) * c.cols, c.cols, nt);
  }
}

// dx of every G-th row, and the workgroup's share of dw and db. Bound by the
// latency of a row's load and two sums, with as many rows in flight as the
// registers allow: 16384 rows of 8192 bf16 in 152 to 172 us, 4.7 to 5.3 TB/s (a call
// 166; 138 for the RMS norm, which keeps db and the sum of g all the same); rows of
// odd width by their single-element accesses (4097 x 1001 fp32: 19 us, and a call
// 29), above 4096 columns also by what the loop over rows spills, 103 to 137 of its
// registers: 4097 x 5001 and 9001 fp32 210 and 340 us a call, 1.0 and 1.1 TB/s.
template <bool IN16, bool DY16, bool P16, bool VEC, int VPT>
__global__ __launch_bounds__(kGradThreads) void norm_grad_kernel(NormCall c, const void* x, const void* dy, void* dx, float* part) {
  __shared__ __attribute__((aligned(16))) float red[4 * kMaxWaves];
  const int nt = static_cast<int>(blockDim.x);
  const float width = static_cast<float>(c.cols);
  int half = 0;
  float dw[VPT][8] = {}, db[VPT][8] = {};
  Row<P16, VEC, VPT> weight;
  weight.load(c.weight, 0, c.cols, nt);
  Row<IN16, VEC, VPT, true> row;
  Row<DY16, VEC, VPT, true> up;
  row.load(x, blockIdx.x * static_cast<int64_t>(c.cols), c.cols, nt);
  up.load(dy, blockIdx.x * static_cast<int64_t>(c.cols), c.cols, nt);
  for (int64_t r = blockIdx.x; r < c.n; r += gridDim.x) {
    weight.hide();
    float h[VPT][8];
    const float inv = standardize(row, h, c.cols, c.eps, c.center, red, half, nt);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float d[8], w[8];
      up.widen(k, d);
      weight.widen(k, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[k][e] = __builtin_fmaf(d[e], h[k][e], dw[k][e]);
        db[k][e] += d[e];
        const float g = d[e] * w[e];
        s[0] = __builtin_fmaf(g, h[k][e], s[0]);
        s[1] += g;
      }
    }
    group_sum<2>(s, red, half, nt);
    const float along = s[0] / width, mean = c.center ? s[1] / width : 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float d[8], w[8];
      up.widen(k, d);
      weight.widen(k, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = (d[e] * w[e] - mean - h[k][e] * along) * inv;
      store8<IN16, VEC>(dx, r * c.cols, k, d, c.cols, nt);
    }
    if (r + gridDim.x < c.n) {
      row.load(x, (r + gridDim.x) * c.cols, c.cols, nt);
      up.load(dy, (r + gridDim.x) * c.cols, c.cols, nt);
    }
  }
  float* mine = part + static_cast<int64_t>(blockIdx.x) * 2 * c.cols;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    store8<false, VEC>(mine, 0, k, dw[k], c.cols, nt);
    if (c.bias) store8<false, VEC>(mine, c.cols, k, db[k], c.cols, nt);
  }
}

// packed <- [prev +] sigma * the sum of the shares, 64 columns a workgroup,
// each by kSlices threads whose sums are added in order. 7 us for 512 shares of
// 8192 columns, 10 for those of 1001: the latency of a chain of loads.
constexpr int kSlices = 16;
struct NormOut {
  const float* prev;
  void* packed;
};

template <bool OUT16>
__global__ __launch_bounds__(kSlices * kWave) void norm_sum_kernel(const float* part, int shares, int cols, NormOut w, NormOut b,
                                                                   float sigma) {
  __shared__ float red[kSlices][kWave];
  const int lane = threadIdx.x % kWave, slice = threadIdx.x / kWave;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kWave + lane;
  const bool second = blockIdx.y == 1;
  float s = 0.0f;
  if (c < cols) {
    const float* p = part + (second ? cols : 0) + c;
#pragma unroll 8
    for (int g = slice; g < shares; g += kSlices) s += p[static_cast<int64_t>(g) * 2 * cols];
  }
  red[slice][lane] = s;
  __syncthreads();
  if (slice || c >= cols) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) s += red[i][lane];
  s *= sigma;
  const NormOut o = second ? b : w;
  if (o.prev) s = o.prev[c] + s;
  if constexpr (OUT16) static_cast<uint16_t*>(o.packed)[c] = static_cast<uint16_t>(bf16_rne(s));
  else static_cast<float*>(o.packed)[c] = s;
}

// ------------------------------------------------------------------ host

constexpr int64_t kNormMaxCols = 16384, kNormMaxRows = int64_t(1) << 31;

struct NormShape {
  int threads, vpt;
  unsigned grid;
};

// The launch of a pass: threads per row, vectors of 8 per thread, and workgroups,
// per_cu threads' worth of them on each of the 256 CUs. 16384 rows of 8192 bf16
// columns: forwards 512 threads with two vectors each and 8192 threads a CU take
// 82 us (4096: 84, 2048: 96; 256 threads with four 84; 1024 with one 110);
// backwards 512 with two and 1024 a CU 161 (1024 with one 216, 256 with four 210;
// 1536 a CU 218), where more workgroups mean more shares to add up. Narrow rows have
// the most of these, 128 threads a row and 2048 shares for 4097 x 1001: their 16 MB
// are written and read beside 41 MB of data (65536 x 64 bf16: 52 us a call, 0.5 TB/s).
NormShape norm_shape(int64_t n, int64_t cols, int vmost, int most, int64_t per_cu) {
  NormShape s{kWave, 1, 0};
  while (s.vpt < vmost && s.threads * 8 * s.vpt < cols) s.vpt *= 2;
  while (s.threads < 512 && s.threads * 8 * s.vpt < cols) s.threads *= 2;
  while (s.vpt < 2 && s.threads * 8 * s.vpt < cols) s.vpt *= 2;
  while (s.threads < most && s.threads * 8 * s.vpt < cols) s.threads *= 2;
  while (s.threads * 8 * s.vpt < cols) s.vpt *= 2;
  s.grid = static_cast<unsigned>(std::min<int64_t>(n, 256 * std::max<int64_t>(1, per_cu / s.threads)));
  return s;
}
NormShape forward_shape(int64_t n, int64_t cols) { return norm_shape(n, cols, 2, kNormThreads, 8192); }
NormShape grad_shape(int64_t n, int64_t cols) { return norm_shape(n, cols, 1, kGradThreads, 1024); }

int64_t grad_work(int64_t n, int64_t cols) { return int64_t(grad_shape(n, cols).grid) * 2 * cols * 4; }

int check_norm(const rs_plan* p, int64_t weight, int64_t bias, int64_t n, const char* who) {
  if (weight < 0 || weight >= p->n || bias < -1 || bias >= p->n || bias == weight)
    return fail(RS_EINVAL, std::string(who) + ": weight and bias are two tensors of the plan (bias -1: none)");
  if (p->t[weight].kind == RS_TILEMAJOR || (bias >= 0 && p->t[bias].kind == RS_TILEMAJOR))
    return fail(RS_EINVAL, std::string(who) + ": a TILEMAJOR tensor is not contiguous");
  if (bias >= 0 && p->t[bias].n != p->t[weight].n)
    return fail(RS_EINVAL, std::string(who) + ": weight and bias differ in size");
  if (n < 0) return fail(RS_EINVAL, std::string(who) + ": negative number of rows");
  if (p->t[weight].n > kNormMaxCols || n >= kNormMaxRows)
    return fail(RS_ERANGE, std::string(who) + ": at most 16384 columns, rows under 2^31");
  return RS_OK;
}

template <typename F>
void by_types(bool a16, bool b16, bool vec, int vpt, F f) {
  auto width = [&](auto a, auto b, auto v) {
    if (vpt == 1) f(a, b, v, std::integral_constant<int, 1>{});
    else if (vpt == 2) f(a, b, v, std::integral_constant<int, 2>{});
    else f(a, b, v, std::integral_constant<int, 4>{});
  };
  auto aligned = [&](auto a, auto b) {
    if (vec) width(a, b, std::true_type{});
    else width(a, b, std::false_type{});
  };
  if (a16 && b16) aligned(std::true_type{}, std::true_type{});
  else if (a16) aligned(std::true_type{}, std::false_type{});
  else if (b16) aligned(std::false_type{}, std::true_type{});
  else aligned(std::false_type{}, std::false_type{});
}

bool f32_or_bf16(int32_t dt) { return dt == RS_F32 || dt == RS_BF16; }

NormCall norm_call(const rs_plan* p, int64_t weight, int64_t bias, const void* gathered, int32_t dt, int64_t n, float eps,
                   int32_t center) {
  const char* g = static_cast<const char*>(gathered);
  return {g + p->t[weight].start * elem_bytes(dt), bias >= 0 ? g + p->t[bias].start * elem_bytes(dt) : nullptr, dt == RS_BF16, n,
          static_cast<int>(p->t[weight].n), eps, center != 0};
}

}  // namespace
}  // namespace rs

using namespace rs;

extern "C" int rs_layer_norm(rs_plan* p, int64_t weight, int64_t bias, const void* gathered, int32_t dt, const void* x,
                             int32_t x_dt, int64_t n_rows, float eps, int32_t center, void* y, int32_t y_dt, void* stream) {
  const char* who = "rs_layer_norm";
  clear_error();
  int st = check_call(p, who);
  if (st == RS_OK) st = check_norm(p, weight, bias, n_rows, who);
  if (st != RS_OK) return st;
  if (!gathered || (n_rows && (!x || !y))) return fail(RS_EINVAL, std::string(who) + ": null argument");
  if (!f32_or_bf16(dt) || !f32_or_bf16(x_dt) || !f32_or_bf16(y_dt)) return fail(RS_EDTYPE, std::string(who) + ": fp32 or bf16");
  if (!(eps >= 0.0f) || !std::isfinite(eps) || (center != 0 && center != 1))
    return fail(RS_EINVAL, std::string(who) + ": eps must be finite and >= 0, center 0 or 1");
  if (!aligned16(gathered) || !aligned16(x) || !aligned16(y))
    return fail(RS_EALIGN, std::string(who) + ": buffers must be 16-byte aligned");
  if (n_rows == 0) return RS_OK;
  const NormCall c = norm_call(p, weight, bias, gathered, dt, n_rows, eps, center);
  const NormShape s = forward_shape(n_rows, c.cols);
  by_types(x_dt == RS_BF16, y_dt == RS_BF16, c.cols % 8 == 0, s.vpt, [&](auto in, auto out, auto vec, auto vpt) {
    hipLaunchKernelGGL((norm_kernel<in.value, out.value, vec.value, vpt.value>), dim3(s.grid),
                       dim3(static_cast<unsigned>(s.threads)), 0, static_cast<hipStream_t>(stream), c, x, y);
  });
  return launched(who);
}

extern "C" int rs_layer_norm_workspace(const rs_plan* p, int64_t weight, int64_t n_rows, int64_t* bytes) {
  const char* who = "rs_layer_norm_workspace";
  clear_error();
  if (!p || !bytes) return fail(RS_EINVAL, std::string(who) + ": null argument");
  const int st = check_norm(p, weight, -1, n_rows, who);
  if (st != RS_OK) return st;
  *bytes = grad_work(n_rows, p->t[weight].n);
  return RS_OK;
}

extern "C" int rs_layer_norm_grad(rs_plan* p, int64_t weight, int64_t bias, const void* gathered, int32_t dt, const void* x,
                                  int32_t x_dt, const void* dy, int32_t dy_dt, int64_t n_rows, float eps, int32_t center,
                                  void* dx, const float* prev, void* packed, int32_t packed_dt, int32_t scale_mode, float scale,
                                  void* work, int64_t work_bytes, void* stream) {
  const char* who = "rs_layer_norm_grad";
  clear_error();
  int st = check_call(p, who);
  if (st == RS_OK) st = check_norm(p, weight, bias, n_rows, who);
  if (st != RS_OK) return st;
  if (!gathered || !packed || (n_rows && (!x || !dy || !dx || !work))) return fail(RS_EINVAL, std::string(who) + ": null argument");
  if (!f32_or_bf16(dt) || !f32_or_bf16(x_dt) || !f32_or_bf16(dy_dt) || !f32_or_bf16(packed_dt))
    return fail(RS_EDTYPE, std::string(who) + ": fp32 or bf16");
  if (!(eps >= 0.0f) || !std::isfinite(eps) || (center != 0 && center != 1))
    return fail(RS_EINVAL, std::string(who) + ": eps must be finite and >= 0, center 0 or 1");
  if (prev == packed && packed_dt != RS_F32)
    return fail(RS_EINVAL, std::string(who) + ": prev may be packed only when packed is fp32");
  if ((scale_mode != RS_SCALE_INV_V && scale_mode != RS_SCALE_GIVEN) || !std::isfinite(scale))
    return fail(RS_EINVAL, std::string(who) + ": bad scale");
  if (!aligned16(gathered) || !aligned16(x) || !aligned16(dy) || !aligned16(dx) || !aligned16(prev) || !aligned16(packed) ||
      !aligned16(work))
    return fail(RS_EALIGN, std::string(who) + ": buffers must be 16-byte aligned");
  const NormCall c = norm_call(p, weight, bias, gathered, dt, n_rows, eps, center);
  const int64_t need = grad_work(n_rows, c.cols);
  if (work_bytes < need)
    return fail(RS_EINVAL, std::string(who) + ": workspace of " + std::to_string(work_bytes) + " bytes, " + std::to_string(need) +
                               " needed");
  const NormShape s = grad_shape(n_rows, c.cols);
  hipStream_t q = static_cast<hipStream_t>(stream);
  if (n_rows)
    by_types(x_dt == RS_BF16, dy_dt == RS_BF16, c.cols % 8 == 0, s.vpt, [&](auto in, auto up, auto vec, auto vpt) {
      constexpr int kVpt = vpt.value > 2 ? 2 : vpt.value;   // norm_shape gives no more
      const dim3 grid(s.grid), threads(static_cast<unsigned>(s.threads));
      if (c.param16)
        hipLaunchKernelGGL((norm_grad_kernel<in.value, up.value, true, vec.value, kVpt>), grid, threads, 0, q, c, x, dy, dx, static_cast<float*>(work));
      else
        hipLaunchKernelGGL((norm_grad_kernel<in.value, up.value, false, vec.value, kVpt>), grid, threads, 0, q, c, x, dy, dx, static_cast<float*>(work));
    });
  auto out = [&](int64_t t) -> NormOut {
    if (t < 0) return {nullptr, nullptr};
    return {prev ? prev + p->t[t].start : nullptr, static_cast<char*>(packed) + p->t[t].start * elem_bytes(packed_dt)};
  };
  const float sigma = scale_mode == RS_SCALE_INV_V ? static_cast<float>(static_cast<double>(scale) / static_cast<double>(p->V)) : scale;
  const dim3 grid(static_cast<unsigned>((c.cols + kWave - 1) / kWave), bias >= 0 ? 2 : 1);
  if (packed_dt == RS_BF16)
    hipLaunchKernelGGL((norm_sum_kernel<true>), grid, dim3(kSlices * kWave), 0, q, static_cast<const float*>(work),
                       static_cast<int>(s.grid), c.cols, out(weight), out(bias), sigma);
  else
    hipLaunchKernelGGL((norm_sum_kernel<false>), grid, dim3(kSlices * kWave), 0, q, static_cast<const float*>(work),
                       static_cast<int>(s.grid), c.cols, out(weight), out(bias), sigma);
  return launched(who);
}
